// The (token, expert) pairs in expert order: a stable counting sort.
//
// Few pairs: one block counts, scans and places them.  Many: count_kernel leaves each
// block's counts in the first E places of its own stretch of `position`; scan_kernel, a warp
// per expert, turns them into the block's first place within the expert and leaves every
// expert's total behind them; place_kernel reads its own stretch before it writes it.  The
// outputs are the only memory used.
// Within a block each warp takes a stretch of its own, and within 32 pairs the rank of a
// pair is the number of lower lanes with the same expert, so the order is the pairs'
// own whatever the timing.
// 512 pairs 2.9 us, a launch; 524288 pairs of 256 experts 13.6 us in three launches, each bound
// by its latency (14.2 before the order of a block was staged too: scattered stores, a lane
// each), where the 6 MB would take 0.9 us.
#include <cstdint>
#include <type_traits>

#include "experts.h"
#include "ptx.cuh"

namespace tn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
// One block takes up to this many pairs by itself (one block, three launches, 256 experts:
// 4096 pairs 5.7, 8.5 us; 8192 pairs 8.7, 8.6).
constexpr int kSinglePairs = 8192;
// Pairs per block beyond that: a block's counts and the experts' totals fit its stretch.
constexpr int kChunk = 2048;
static_assert(kChunk >= 2 * kMaxExperts, "a block's counts and the totals fit its stretch of the output");
constexpr int kCountThreads = 512;
constexpr int kPlaceWarps = 16;
constexpr int kSingleWarps = 32;
constexpr int kScanWarps = 8;

// Pairs of block b, from pair b * kChunk on.  The last block takes the rest, so every block has
// at least kChunk.  Places within a block are counted from its first pair: up to 2^31 - 1 pairs
// fit an int, a step past the last of them does not.
__device__ __forceinline__ int block_pairs(int b, int blocks, int n) { return b == blocks - 1 ? n - b * kChunk : kChunk; }

__global__ void __launch_bounds__(kCountThreads) count_kernel(const int32_t* ids, int32_t* position, int n, int E, int blocks) {
    __shared__ int count[kMaxExperts];
    for (int e = threadIdx.x; e < E; e += kCountThreads) count[e] = 0;
    griddep_launch_dependents();
    griddep_wait();
    __syncthreads();
    const int b = blockIdx.x, begin = b * kChunk, own = block_pairs(b, blocks, n);
#pragma unroll 8
    for (int i = threadIdx.x; i < own; i += kCountThreads) {
        const unsigned e = static_cast<unsigned>(ids[begin + i]);
        if (e < static_cast<unsigned>(E)) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kCountThreads) position[begin + e] = count[e];
}

// Exclusive scan of v over the block's threads (kThreads of them); *total: the sum.
template <int kThreads, class Sum>
__device__ __forceinline__ Sum block_scan(Sum v, Sum* warp_sums, Sum* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sum incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum u = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        Sum s = lane < kThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sum u = __shfl_up_sync(kFull, s, o);
            if (lane >= o) s += u;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    *total = warp_sums[31];
    return incl - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// One warp per expert: its counts of 32 blocks at a time, scanned; then its total to every block.
__global__ void __launch_bounds__(kScanWarps * 32) scan_kernel(int32_t* position, int E, int blocks) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, e = blockIdx.x * kScanWarps + (threadIdx.x >> 5);
    if (e >= E) return;
    int sum = 0;
    constexpr int U = 8;  // counts in flight per lane
    for (int b0 = 0; b0 < blocks; b0 += 32 * U) {
        int c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * 32 + lane;
            c[u] = b < blocks ? position[b * kChunk + e] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = b0 + u * 32 + lane;
            int incl = c[u];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += v;
            }
            if (b < blocks) position[b * kChunk + e] = sum + incl - c[u];
            sum += __shfl_sync(kFull, incl, 31);
        }
    }
    for (int b = lane; b < blocks; b += 32) position[b * kChunk + E + e] = sum;
}

// The lanes with this lane's v < 2^bits, by a ballot per bit: ~50 instructions where a match
// instruction holds the SM ~55 cycles (8192 pairs in one
// block: 14.4 us with match, 8.7 without it and with the order staged).
__device__ __forceinline__ unsigned lanes_alike(unsigned v, int bits) {
    unsigned same = kFull;
#pragma unroll
    for (int b = 0; b < 11; ++b) {
        static_assert(kMaxExperts < 1 << 11, "bits of an expert or of none");
        if (b < bits) {
            const bool set = (v >> b) & 1u;
            const unsigned lanes = __ballot_sync(kFull, set);
            same &= set ? lanes : ~lanes;
        }
    }
    return same;
}

// Places the block's pairs, PER groups of 32 of them per warp at most.  count[w][e]: first
// the pairs of expert e in warp w's stretch, then the place of the first of them within the
// block's own order.  SINGLE: the block holds all pairs.
template <bool SINGLE, int WARPS, int PER>
__global__ void __launch_bounds__(WARPS * 32)
    place_kernel(const int32_t* ids, int32_t* offsets, int32_t* order, int32_t* position, int n, int E, int blocks) {
    extern __shared__ int count[];  // [WARPS][E]
    // scanned together: pairs of an expert in all blocks << 16 | in this one (one block: these alone)
    using Sum = std::conditional_t<SINGLE, int, long long>;
    constexpr int kThreads = WARPS * 32, kPairs = PER * kThreads;
    static_assert(SINGLE || kPairs < 1 << 16, "the block's own sums fit their bits");
    __shared__ Sum warp_sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < WARPS * E; i += kThreads) count[i] = 0;
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x, begin = SINGLE ? 0 : b * kChunk, pairs = SINGLE ? n : block_pairs(b, blocks, n);
    const int per = ((pairs + kThreads - 1) / kThreads) * 32;  // pairs per warp, whole groups of 32
    const int w0 = warp * per, w1 = min(pairs, w0 + per);
    int* row = count + warp * E;
    int* shift = count + WARPS * E;                  // not SINGLE: [E], from the block's order to all blocks'
    int* sorted = shift + (SINGLE ? 0 : E);          // [n or kPairs], the pairs in the block's order
    int* target = sorted + kPairs;                   // not SINGLE: [kPairs], their places
    const int bits = 32 - __clz(E);                  // of 0 .. E
    unsigned id[PER];
    int at[PER];  // place within the warp's pairs of the expert
#pragma unroll
    for (int j = 0; j < PER; ++j) id[j] = w0 + j * 32 + lane < w1 ? static_cast<unsigned>(ids[begin + w0 + j * 32 + lane]) : 0xffffffffu;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (w0 + j * 32 >= w1) break;
        const bool in = id[j] < static_cast<unsigned>(E);
        const unsigned same = lanes_alike(in ? id[j] : static_cast<unsigned>(E), bits);
        at[j] = in ? row[id[j]] + __popc(same & ((1u << lane) - 1u)) : 0;
        __syncwarp();
        if (in && lane == 31 - __clz(same)) row[id[j]] = at[j] + 1;
        __syncwarp();
    }
    __syncthreads();
    // places of the experts, then of each warp's first pair of them
    Sum last = 0;  // pairs of all experts
    for (int e0 = 0; e0 < E; e0 += kThreads) {
        const int e = e0 + threadIdx.x;
        int before = 0;
        Sum total = 0;
        if (e < E) {
            for (int w = 0; w < WARPS; ++w) total += count[w * E + e];
            if (!SINGLE) {
                before = position[begin + e];
                total += static_cast<Sum>(position[begin + E + e]) << (SINGLE ? 0 : 16);
            }
        }
        Sum sum;
        const Sum scan = last + block_scan<kThreads>(total, warp_sums, &sum);
        __syncthreads();  // warp_sums is used again
        if (e < E) {
            const int first = static_cast<int>(SINGLE ? scan : scan >> 16);
            int next = static_cast<int>(SINGLE ? scan : scan & 0xffff);
            if (b == 0) offsets[e] = first;
            if (!SINGLE) shift[e] = first + before - next;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const int c = count[w * E + e];
                count[w * E + e] = next;
                next += c;
            }
        }
        last += sum;
    }
    const int all = static_cast<int>(SINGLE ? last : last >> 16), mine = static_cast<int>(SINGLE ? last : last & 0xffff);
    if (b == 0 && threadIdx.x == 0) offsets[E] = all;
    __syncthreads();  // the block's stretch is read before it is written
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = w0 + j * 32 + lane;
        if (i < w1) {
            int to = -1;
            if (id[j] < static_cast<unsigned>(E)) {
                const int own = row[id[j]] + at[j];
                to = SINGLE ? own : own + shift[id[j]];
                sorted[own] = begin + i;
                if (!SINGLE) target[own] = to;
            }
            position[begin + i] = to;
        }
    }
    // The order goes through shared memory: a store whose lanes are scattered takes a cycle per
    // lane of the SM's one store path, one of runs (a run is a block's pairs of one expert) few.
    __syncthreads();
    for (int i = threadIdx.x; i < mine; i += kThreads) order[SINGLE ? i : target[i]] = sorted[i];
    for (int i = min(max(all - begin, 0), pairs) + static_cast<int>(threadIdx.x); i < pairs; i += kThreads) order[begin + i] = -1;
}

}  // namespace
}  // namespace tn

extern "C" gemm_status_t expert_group(int64_t T, int64_t top_k, int64_t E, const int32_t* ids, int32_t* offsets,
                                      int32_t* order, int32_t* position, cudaStream_t stream) {
    using namespace tn;
    if (T < 0 || top_k < 1 || E < 1 || E > kMaxExperts || T >= (int64_t(1) << 31) || top_k >= (int64_t(1) << 31) ||
        T * top_k >= (int64_t(1) << 31))
        return GEMM_ERR_INVALID_ARG;
    if (offsets == nullptr || (T > 0 && (ids == nullptr || order == nullptr || position == nullptr))) return GEMM_ERR_INVALID_ARG;
    if (!aligned_to(ids, 4) || !aligned_to(offsets, 4) || !aligned_to(order, 4) || !aligned_to(position, 4))
        return GEMM_ERR_ALIGNMENT;
    const uint64_t pairs = uint64_t(T) * top_k * 4, off = uint64_t(E + 1) * 4;
    if (T > 0 && (overlaps(ids, pairs, offsets, off) || overlaps(ids, pairs, order, pairs) || overlaps(ids, pairs, position, pairs) ||
                  overlaps(order, pairs, position, pairs) || overlaps(order, pairs, offsets, off) ||
                  overlaps(position, pairs, offsets, off)))
        return GEMM_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    const gemm_status_t st = device_info(&dev, &sms);
    if (st != GEMM_OK) return st;
    const int n = static_cast<int>(T * top_k), e = static_cast<int>(E);
    constexpr int kSinglePer = kSinglePairs / (kSingleWarps * 32);
    constexpr int kPlacePer = (2 * kChunk + kPlaceWarps * 32 - 1) / (kPlaceWarps * 32);  // the last block takes the rest
    if (n <= kSinglePairs) {
        auto kernel = place_kernel<true, kSingleWarps, kSinglePer>;
        const size_t smem = sizeof(int) * (kSingleWarps * E + n);
        if (allow_smem(kernel, sizeof(int) * (kSingleWarps * kMaxExperts + kSinglePairs), dev) != cudaSuccess) return GEMM_ERR_CUDA;
        return launch_pdl(kernel, dim3(1), dim3(kSingleWarps * 32), smem, stream, ids, offsets, order, position, n, e, 1) == cudaSuccess
                   ? GEMM_OK
                   : GEMM_ERR_CUDA;
    }
    const int blocks = n / kChunk;
    auto place = place_kernel<false, kPlaceWarps, kPlacePer>;
    constexpr int kPlacePairs = kPlacePer * kPlaceWarps * 32;
    const auto place_smem = [](int64_t experts) { return sizeof(int) * ((kPlaceWarps + 1) * experts + 2 * kPlacePairs); };
    if (allow_smem(place, place_smem(kMaxExperts), dev) != cudaSuccess) return GEMM_ERR_CUDA;
    if (launch_pdl(count_kernel, dim3(blocks), dim3(kCountThreads), 0, stream, ids, position, n, e, blocks) != cudaSuccess ||
        launch_pdl(scan_kernel, dim3((e + kScanWarps - 1) / kScanWarps), dim3(kScanWarps * 32), 0, stream, position, e, blocks) != cudaSuccess ||
        launch_pdl(place, dim3(blocks), dim3(kPlaceWarps * 32), place_smem(E), stream, ids, offsets, order, position,
                   n, e, blocks) != cudaSuccess)
        return GEMM_ERR_CUDA;
    return GEMM_OK;
}
