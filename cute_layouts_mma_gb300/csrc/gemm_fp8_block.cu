// Entry points and launchers of the block-scaled FP8 products, plain and grouped.
#include <cstdint>

#include "gemm_fp8_block_kernel.cuh"
#include "launch_kernel.cuh"

namespace tn {

// Device-side record of an abandoned launch (a bounded wait ran out).
static __device__ unsigned int g_err_fp8_block;

namespace {

std::atomic<uintptr_t> g_err_addr[kMaxDevices];

struct Operands {
    int64_t rows_a, rows_b;  // rows of A, rows of B over all experts
    const void *A, *B;
};

template <class Cfg>
gemm_status_t run(const Operands& o, Fp8Params p, cudaStream_t stream, int sms, int dev) {
    auto kernel = gemm_fp8_block_kernel<Cfg>;
    CUtensorMap ta, tb, tc, td;
    constexpr uint32_t kRowBox = 128, kColBox = Cfg::BN_CTA;
    if (!make_tma_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.A, p.K, o.rows_a, p.K, 128, Cfg::kSwap ? kColBox : kRowBox, 128) ||
        !make_tma_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.B, p.K, o.rows_b, p.K, 128, Cfg::kSwap ? kRowBox : kColBox, 128))
        return GEMM_ERR_CUDA;
    // C and D in boxes of 32 rows x 128 bytes (the swapped form takes none)
    tc = td = ta;
    auto box_map = [&](CUtensorMap* map, const void* base) {
        return make_tma_2d(map, p.f32_out ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, p.N, o.rows_a,
                           static_cast<uint64_t>(p.N) * (p.f32_out ? 4 : 2), p.f32_out ? 32 : 64, 32, 128);
    };
    if (!Cfg::kSwap && (!box_map(&td, p.D) || (p.C != nullptr && !box_map(&tc, p.C)))) return GEMM_ERR_CUDA;
    p.err = device_symbol(g_err_fp8_block, g_err_addr, dev);
    if (p.err == nullptr) return GEMM_ERR_CUDA;

    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.blockDim = dim3(Cfg::THREADS);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    auto cluster = [&](int n) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(n);
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    };
    if (Cfg::PAIR == 2) cluster(2);
    static std::atomic<int> seen_units[kMaxDevices];  // resident CTAs, or CTA pairs
    int units = seen_units[dev].load(std::memory_order_acquire);
    if (units == 0) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) != cudaSuccess) return GEMM_ERR_CUDA;
        if (Cfg::kRegSplit) {
            // the promotion warps' registers come from what the launch holds and the others give up
            // (another count, at which they would wait for ever, already fails the build: build.py)
            cudaFuncAttributes fa{};
            if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs != Cfg::kRegsLaunch) return GEMM_ERR_CUDA;
        }
        units = sms;
        if (Cfg::PAIR == 2) {
            cfg.gridDim = dim3(static_cast<unsigned>(2 * (sms / 2)));
            if (cudaOccupancyMaxActiveClusters(&units, kernel, &cfg) != cudaSuccess) return GEMM_ERR_CUDA;
            if (units <= 0) units = sms / 2;
        }
        seen_units[dev].store(units, std::memory_order_release);
    }
    p.num_m = static_cast<int>((o.rows_a + Cfg::TM - 1) / Cfg::TM);
    p.num_n = static_cast<int>((int64_t(p.N) + Cfg::TN - 1) / Cfg::TN);
    const long long tiles = static_cast<long long>(p.num_m) * p.num_n;
    if (tiles > 0x7fffffffLL / 8) return GEMM_ERR_INVALID_ARG;
    const long long row = static_cast<long long>(p.nkb) * 128;
    p.raster_group = dispatch::raster_group(p.num_m, p.num_n, units, Cfg::TM * row, Cfg::TN * row);
    p.split = 1;
    if constexpr (Cfg::kSplit) {
        // CTAs per tile: the most, of 2, 4 and 8, that leaves each kSplitShare blocks of K, one
        // CTA per SM and every cluster resident, from kSplitBlocks blocks of K on: joining the
        // partial sums costs 1 to 2 us.  Without and with (us): 512 x 1024 x 4096 11.1, 9.3 and
        // x 2048 7.2, 8.4; 128 x 1024 x 4096 10.8, 8.2 and x 2048 7.0, 7.1; swapped, with less
        // to join, 16 x 1024 x 2048 5.5, 4.4 and x 1024 4.1, 4.3.  Shares of 2, 4 and 8 blocks
        // are within 3 % from 4096 on; 16 are slower (128 x 1024 x 4096 9.3).
        constexpr int kSplitShare = 4, kSplitBlocks = Cfg::kSwap ? 16 : 32;
        static std::atomic<int> resident[kMaxDevices][4];  // clusters of 2^i CTAs resident at once; -1: none
        for (int i = 1; i <= 3; ++i) {
            const int ways = 1 << i;
            if (p.nkb < kSplitBlocks || p.nkb < ways * kSplitShare || tiles * ways > sms || !Cfg::split_fits(ways)) break;
            int n = resident[dev][i].load(std::memory_order_acquire);
            if (n == 0) {
                cudaLaunchAttribute a[1];
                a[0].id = cudaLaunchAttributeClusterDimension;
                a[0].val.clusterDim.x = static_cast<unsigned>(ways);
                a[0].val.clusterDim.y = 1;
                a[0].val.clusterDim.z = 1;
                cudaLaunchConfig_t c = cfg;
                c.attrs = a;
                c.numAttrs = 1;
                c.gridDim = dim3(static_cast<unsigned>(sms / ways * ways));
                if (cudaOccupancyMaxActiveClusters(&n, kernel, &c) != cudaSuccess) {
                    (void)cudaGetLastError();
                    n = 0;
                }
                if (n == 0) n = -1;
                resident[dev][i].store(n, std::memory_order_release);
            }
            if (tiles > n) break;
            p.split = ways;
        }
    }
    if (Cfg::kSplit && p.split > 1) {
        cluster(p.split);
        cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split));
    } else {
        // grouped: the tiles are counted on the device; every unit looks for some
        cfg.gridDim = dim3(static_cast<unsigned>((Cfg::kGrouped || tiles > units ? units : tiles) * Cfg::PAIR));
    }
    add_pdl(cfg);
    return cudaLaunchKernelEx(&cfg, kernel, ta, tb, tc, td, p) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// mode, CTAs per tile, columns, stages, k-blocks per stage, accumulators, promotion warps, grouped
using RowsN128 = Fp8Config<MODE_ROWS, 1, 128, 5, 1, 4, 8, false>;
using BothN128 = Fp8Config<MODE_BOTH, 1, 128, 5, 1, 4, 8, false>;
using GroupedN128 = Fp8Config<MODE_ROWS, 1, 128, 5, 1, 4, 8, true>;
using RowsPair = Fp8Config<MODE_ROWS, 2, 256, 4, 1, 2, 8, false>;
using BothPair = Fp8Config<MODE_BOTH, 2, 256, 4, 1, 2, 8, false>;
using GroupedSingle = Fp8Config<MODE_ROWS, 1, 256, 3, 1, 2, 8, true>;
using GroupedPair = Fp8Config<MODE_ROWS, 2, 256, 4, 1, 2, 8, true>;
// Few rows of A: swapped, so that the weights stream through the MMA's 128 rows and only
// BN columns are summed and stored; two blocks of K per stage halve the waits per byte.
template <bool GROUPED>
using Swap16 = Fp8Config<MODE_SWAP, 1, 16, 5, 2, 5, 4, GROUPED>;
template <bool GROUPED>
using Swap32 = Fp8Config<MODE_SWAP, 1, 32, 5, 2, 5, 4, GROUPED>;
template <bool GROUPED>
using Swap64 = Fp8Config<MODE_SWAP, 1, 64, 4, 2, 4, 4, GROUPED>;

// CTA pairs with 256 x 256 tiles, or single CTAs with 128 x 128: the smaller of rounds of tiles
// x (a tile's blocks x a block's time + a tile's own time), fitted to measurements in units of
// ~8 ns (a scale per row and column: ~11).  A block takes a pair 40 and a single CTA 30 units
// (50 and 30) for a quarter of the pair's work, so pairs win once both are busy: single, pair (us)
// 1024 x 4096 x 4096 20.5, 17.3 (25.0, 23.9); 4096^3 62, 54 (80, 81).  Pairs read half as much
// per product, which tells where rows that are no multiple of 128 bytes spread over more lines:
// 4096 x 4096 x 4112 90, 61 (101, 85).  Their tiles' start and store are hidden less:
// 4096 x 4096 x 512 13.3, 14.6 (19.4, 22.2); and they are coarser: 1024 x 2048 x 8192 20, 27
// (24, 40); 2560 x 2560 x 4096 28.5, 29.1 (36, 43).
bool use_pairs(int64_t M, int64_t N, int64_t K, int sms, bool both) {
    auto rounds = [](int64_t m, int64_t n, int64_t units) { return (m * n + units - 1) / units; };
    const int64_t pair = rounds((M + 255) / 256, (N + 255) / 256, sms / 2), single = rounds((M + 127) / 128, (N + 127) / 128, sms);
    const int64_t nkb = (K + kFp8Block - 1) / kFp8Block;
    const bool whole = K % kFp8Block == 0;
    const int block_pair = both ? (whole ? 50 : 51) : (whole ? 40 : 44), block_single = whole ? 30 : both ? 37 : 43;
    return pair * (nkb * block_pair + (both ? 200 : 150)) < single * (nkb * block_single + (both ? 60 : 30));
}

bool sizes_ok(int64_t M, int64_t N, int64_t K) {
    constexpr int64_t kLimit = int64_t(1) << 31;
    return M >= 0 && M < kLimit && N >= 1 && N < kLimit && K >= 1 && K < kLimit;
}

// Rows of A, and of B over all experts, of a grouped product: an expert's tiles begin at any row
// and the last one reaches up to 255 rows past its end, within an int still.
constexpr int64_t kMaxGroupedRows = (int64_t(1) << 31) - 512;

}  // namespace

unsigned int read_clear_error_fp8_block() { return read_clear_word(g_err_fp8_block); }

}  // namespace tn

extern "C" {

gemm_status_t gemm_fp8_block(int64_t M, int64_t N, int64_t K, const void* A, const float* SFA, const void* B,
                             const float* SFB, int scales, const void* C, void* D, int out_dtype, cudaStream_t stream) {
    using namespace tn;
    if (!sizes_ok(M, N, K) || (scales != FP8_ROWS && scales != FP8_TILES) ||
        (out_dtype != GEMM_DT_BF16 && out_dtype != GEMM_DT_F32))
        return GEMM_ERR_INVALID_ARG;
    if (K % 16 != 0 || N % 8 != 0) return GEMM_ERR_ALIGNMENT;
    if (M == 0) return GEMM_OK;
    if (A == nullptr || SFA == nullptr || B == nullptr || SFB == nullptr || D == nullptr) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(A) || !aligned16(B) || !aligned16(C) || !aligned16(D) || !aligned_to(SFA, 4) || !aligned_to(SFB, 4))
        return GEMM_ERR_ALIGNMENT;
    const uint64_t nkb = uint64_t(K + kFp8Block - 1) / kFp8Block;
    const uint64_t dbytes = uint64_t(M) * N * (out_dtype == GEMM_DT_F32 ? 4 : 2);
    const uint64_t sfb = 4 * nkb * (scales == FP8_ROWS ? N : (N + kFp8Block - 1) / kFp8Block);
    if (overlaps(D, dbytes, A, uint64_t(M) * K) || overlaps(D, dbytes, B, uint64_t(N) * K) || overlaps(D, dbytes, SFA, 4 * nkb * M) ||
        overlaps(D, dbytes, SFB, sfb) || (C != nullptr && C != D && overlaps(C, dbytes, D, dbytes)))
        return GEMM_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    const gemm_status_t st = device_info(&dev, &sms);
    if (st != GEMM_OK) return st;
    Fp8Params p{};
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.nkb = static_cast<int>(nkb);
    p.sfa = SFA;
    p.sfb = SFB;
    p.C = C;
    p.D = D;
    p.f32_out = out_dtype == GEMM_DT_F32;
    const Operands o{M, N, A, B};
    // Few rows, swapped: 16, 32, 64 columns and not swapped (us), 16 x 16384 x 8192 23.8, 24.0,
    // 24.6, 26.4; 24 rows 39.8, 24.0, 24.7, 26.5; 48 rows 38.8, 40.2, 25.2, 26.5; 96 rows (64
    // columns twice) 42.4, 26.9; 16 x 1024 x 8192 5.9, 6.3, 7.1, 8.9.
    if (scales == FP8_TILES && M <= 64) {
        if (M <= 16) return run<Swap16<false>>(o, p, stream, sms, dev);
        if (M <= 32) return run<Swap32<false>>(o, p, stream, sms, dev);
        return run<Swap64<false>>(o, p, stream, sms, dev);
    }
    if (use_pairs(M, N, K, sms, scales == FP8_ROWS))
        return scales == FP8_ROWS ? run<BothPair>(o, p, stream, sms, dev) : run<RowsPair>(o, p, stream, sms, dev);
    return scales == FP8_ROWS ? run<BothN128>(o, p, stream, sms, dev) : run<RowsN128>(o, p, stream, sms, dev);
}

gemm_status_t gemm_fp8_block_grouped(int64_t R, int64_t N, int64_t K, int64_t E, const void* A, const float* SFA,
                                     const void* B, const float* SFB, const int32_t* offsets, void* D,
                                     cudaStream_t stream) {
    using namespace tn;
    if (!sizes_ok(R, N, K) || E < 1 || E > kMaxExperts || R > kMaxGroupedRows || E * N > kMaxGroupedRows) return GEMM_ERR_INVALID_ARG;
    if (K % 16 != 0 || N % 8 != 0) return GEMM_ERR_ALIGNMENT;
    if (R == 0) return GEMM_OK;
    if (A == nullptr || SFA == nullptr || B == nullptr || SFB == nullptr || offsets == nullptr || D == nullptr) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(A) || !aligned16(B) || !aligned16(D) || !aligned_to(SFA, 4) || !aligned_to(SFB, 4) || !aligned_to(offsets, 4))
        return GEMM_ERR_ALIGNMENT;
    const uint64_t nkb = uint64_t(K + kFp8Block - 1) / kFp8Block, dbytes = uint64_t(R) * N * 2;
    const uint64_t sfb = 4 * nkb * E * ((N + kFp8Block - 1) / kFp8Block);
    if (overlaps(D, dbytes, A, uint64_t(R) * K) || overlaps(D, dbytes, B, uint64_t(E) * N * K) || overlaps(D, dbytes, SFA, 4 * nkb * R) ||
        overlaps(D, dbytes, SFB, sfb) || overlaps(D, dbytes, offsets, 4 * (E + 1)))
        return GEMM_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    const gemm_status_t st = device_info(&dev, &sms);
    if (st != GEMM_OK) return st;
    Fp8Params p{};
    p.M = static_cast<int>(R);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.nkb = static_cast<int>(nkb);
    p.sfa = SFA;
    p.sfb = SFB;
    p.offsets = offsets;
    p.experts = static_cast<int>(E);
    p.D = D;
    const Operands o{R, E * N, A, B};
    // By the rows an expert has on average.  Swapped, 16, 32 and 64 columns, singles of 128 x 128
    // and 128 x 256, pairs (us; 64 experts of 4096 x 2048, unevenly loaded):
    //     8 rows   84   84   83   88   --  119        128 rows  346  190  141  114  106  133
    //    16        86   84   83   88   87  123        256       651  352  243  174  155  174
    //    40       125   91   84   90   --  126        512        --   --   --  301  267  267
    //    64       183  113   91   94   97  127       1024        --   --   --   --  489  475
    // (8 experts of 8192 x 4096: 12 rows 50, 46, 47, 52; 64 rows 91, 58, 53, 51, 51, 68; 512 rows
    // 145, 127, 138; 1024 rows 229, 213 the last two.)  Pairs read a third less per product but
    // leave 128 rows of an expert's last tile empty, on average, where 128 rows leave 64.
    // Where even the 128 x 128 tiles fit on the SMs at one time, they take 0.6 of the time of
    // those of 128 x 256.
    const int64_t rows = R / E, cols = (N + 127) / 128;
    if (rows <= 8) return run<Swap16<true>>(o, p, stream, sms, dev);
    if (rows <= 16) return run<Swap32<true>>(o, p, stream, sms, dev);
    if (rows <= 64) return run<Swap64<true>>(o, p, stream, sms, dev);
    if ((R / 128 + E) * cols <= sms) return run<GroupedN128>(o, p, stream, sms, dev);
    return rows < 768 ? run<GroupedSingle>(o, p, stream, sms, dev) : run<GroupedPair>(o, p, stream, sms, dev);
}

}  // extern "C"
