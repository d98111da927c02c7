// FP8 E4M3 quantisation with a scale per block of 128: along rows (with a gather of the
// rows), along columns with the output transposed, and in tiles of 128 x 128.
//
// All forms read X once and write one byte per element; they are bound by HBM (columns of 8200
// x 8192 bf16: 204 MB in 38.6 us, 79 % of the copy bandwidth; tiles 32, transposed tiles 35) and, gathered rows, which come
// from L2, by the SM's own work (32768 rows of 4096 out of 4096: 268 MB read there and 139 MB
// written in 40.6 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>
#include <type_traits>

#include "experts.h"
#include "ptx.cuh"

namespace tn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kFp8Max = 448.0f;                       // largest E4M3 value
constexpr float kFloor = 7.888609052210118e-31f;        // 2^-100: 448 / it is finite
constexpr int kThreads = 256;

// Eight consecutive elements of X as they are in memory: 16 bytes, or 32 for fp32.
template <class T>
struct alignas(16) Eight {
    T v[8];
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ void clear(Eight<T>& x) {
    uint4* w = reinterpret_cast<uint4*>(&x);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(x) / 16); ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
}

// X through the read-only path, in 16-byte loads.  (No eviction hint: gathered rows are read once
// per row that asks for them, and that is from L2.)
template <class T>
__device__ __forceinline__ void load_eight(Eight<T>& x, const T* p) {
    uint4* w = reinterpret_cast<uint4*>(&x);
    const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(x) / 16); ++i) w[i] = __ldg(q + i);
}

// Largest magnitude, NaN left out (fmaxf takes the other operand).
template <class T>
__device__ __forceinline__ float amax8(const Eight<T>& x) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(to_f32(x.v[i])));
    return a;
}

__device__ __forceinline__ float block_scale(float amax) { return fmaxf(amax, kFloor) / kFp8Max; }
__device__ __forceinline__ float block_factor(float amax) { return kFp8Max / fmaxf(amax, kFloor); }

// Two values to E4M3 codes, to nearest even; rounding past 448 saturates, NaN stays NaN.
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) { return codes2(a, b) | codes2(c, d) << 16; }

struct RowsParams {
    const void* X;
    const int32_t* index;
    uint8_t* Q;
    float* SF;
    int64_t M, ld, R;
    uint32_t K;  // below 2^31: a segment's end, and the step to the next, fit 32 bits without a sign
    int blocks;
    int index_div;
};

// Largest magnitude of eight 16-bit values, two at a time; NaN is left out.
template <class T2>
__device__ __forceinline__ float amax8_packed(const uint4& w) {
    const uint32_t u[4] = {w.x & 0x7fff7fffu, w.y & 0x7fff7fffu, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu};
    const T2* h = reinterpret_cast<const T2*>(u);
    const T2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    const float lo = to_f32(m.x), hi = to_f32(m.y);
    // both halves of a pair may be NaN
    return fmaxf(fmaxf(lo, hi), 0.0f);
}
__device__ __forceinline__ float amax_of(const Eight<float>& x) { return amax8(x); }
__device__ __forceinline__ float amax_of(const Eight<__nv_bfloat16>& x) {
    return amax8_packed<__nv_bfloat162>(*reinterpret_cast<const uint4*>(&x));
}
__device__ __forceinline__ float amax_of(const Eight<__half>& x) { return amax8_packed<__half2>(*reinterpret_cast<const uint4*>(&x)); }

// Two values times a factor in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float f) {
    float2 r;
    asm("{\n\t.reg .b64 a, f, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 f, {%4, %4};\n\tmul.rn.f32x2 r, a, f;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(f));
    return r;
}

// Blocks of 1 x 128.  A warp takes U pieces of 256 elements of one row at a time, each lane
// eight elements of each piece (so sixteen lanes a block), all loads issued together.  The
// 2U block maxima are reduced in about U + 3 shuffles by halving: with each exchange a
// lane keeps half of its pieces, so that in the end lanes hold one block each, and the two
// divisions of a block are made once, by the lanes that hold it, instead of by all of them.
// Rows lie along grid.x and their segments of U pieces along grid.y, so that no index is
// divided.  Bound by instructions next to HBM: 23 per element and 117 us with a maximum
// and a division per lane, 7 and 41 us so (32768 x 4096 bf16 gathered).
template <class T, int U>
__global__ void __launch_bounds__(kThreads) rows_kernel(const RowsParams p) {
    static_assert(U == 1 || U == 2 || U == 4 || U == 8, "pieces per segment");
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, l = lane & 15;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= p.R) return;
    int64_t src = row;
    if (p.index != nullptr) {
        const int at = p.index[row];
        src = at < 0 ? -1 : at / p.index_div;
        if (src >= p.M) src = -1;
    }
    const T* x_row = static_cast<const T*>(p.X) + (src < 0 ? 0 : src * p.ld);
    uint8_t* q_row = p.Q + row * p.K;
    auto segment = [&](const uint32_t seg, auto whole) {
        constexpr bool kWhole = decltype(whole)::value;  // every element of the segment is there
        const uint32_t k0 = seg * (U * 256) + lane * 8;
        Eight<T> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!kWhole) clear(x[u]);
            if (kWhole || (src >= 0 && k0 + u * 256 < p.K)) load_eight(x[u], x_row + k0 + u * 256);
        }
        float a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] = amax_of(x[u]);
        // halving: with `o` lanes to go and n pieces held, a lane keeps the half its bit names
        int piece = 0;  // the piece this lane ends with
#pragma unroll
        for (int o = 8, n = U; o > 0; o >>= 1) {
            if (n > 1) {
                const bool up = (l & o) != 0;
                n >>= 1;
                piece = 2 * piece + (up ? 1 : 0);
#pragma unroll
                for (int i = 0; i < U / 2; ++i)
                    if (i < n) {
                        const float give = up ? a[i] : a[i + n], keep = up ? a[i + n] : a[i];
                        a[i] = fmaxf(keep, __shfl_xor_sync(kFull, give, o));
                    }
            } else {
                a[0] = fmaxf(a[0], __shfl_xor_sync(kFull, a[0], o));
            }
        }
        const float factor = block_factor(a[0]);
        const int block = static_cast<int>(seg * (U * 2)) + 2 * piece + (lane >> 4);
        // of the 16 / U lanes that hold a block, the first writes its scale
        if ((l & (16 / U - 1)) == 0 && block < p.blocks) p.SF[row * p.blocks + block] = block_scale(a[0]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // piece u lies with the lane of its half-warp whose upper bits are u
            const float f = __shfl_sync(kFull, factor, (lane & 16) + u * (16 / U));
            float2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = mul2(make_float2(to_f32(x[u].v[2 * i]), to_f32(x[u].v[2 * i + 1])), f);
            if (kWhole || k0 + u * 256 < p.K)
                *reinterpret_cast<uint2*>(q_row + k0 + u * 256) =
                    make_uint2(codes4(v[0].x, v[0].y, v[1].x, v[1].y), codes4(v[2].x, v[2].y, v[3].x, v[3].y));
        }
    };
    for (uint32_t seg = blockIdx.y; seg * (U * 256) < p.K; seg += gridDim.y) {
        if (src >= 0 && (seg + 1) * (U * 256) <= p.K)
            segment(seg, std::true_type{});
        else
            segment(seg, std::false_type{});
    }
}

struct TileParams {
    const void* X;
    uint8_t* Q;
    float* SF;
    int64_t ld;
    int M, K;
    int64_t pitch;     // bytes per row of Q
    int64_t sf_pitch;  // scales per row of SF
};

// One 128 x 128 tile of X per block of 256 threads.  Thread (g, c) holds the eight columns
// 8c .. 8c+7 of rows 4g .. 4g+3 and 64 + 4g .. 64 + 4g+3, so that four rows of a column are
// one word of the transposed output.  The transposed codes pass through shared memory:
// column n's word w (rows 4w .. 4w+3) lies at word w ^ 2 (n / 8) of its 128-byte line, which
// keeps both the writes of a warp (2 g x 16 c) and its reads free of bank conflicts.
template <class T, int LAYOUT>
__global__ void __launch_bounds__(kThreads) tile_kernel(const TileParams p) {
    constexpr bool kTransposed = LAYOUT != FP8_TILES;
    constexpr bool kColumns = LAYOUT == FP8_COLS;  // a scale per column of the tile, not per tile
    __shared__ __align__(16) uint32_t codes[kTransposed ? 128 * 32 : 1];
    __shared__ float part[8][128];
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
    const int m0 = static_cast<int>(blockIdx.y) * 128, k0 = static_cast<int>(blockIdx.x) * 128;
    Eight<T> x[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = m0 + h * 64 + 4 * g + i, k = k0 + 8 * c;
            clear(x[h][i]);
            if (m < p.M && k < p.K) load_eight(x[h][i], static_cast<const T*>(p.X) + m * p.ld + k);
        }
    float a[8];  // kColumns: maximum of each of the thread's columns; else a[0], the thread's
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        a[j] = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) a[j] = fmaxf(a[j], fabsf(to_f32(x[h][i].v[j])));
    }
    if constexpr (kColumns) {
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = fmaxf(a[j], __shfl_xor_sync(kFull, a[j], 16));
        if (lane < 16) {
#pragma unroll
            for (int j = 0; j < 8; j += 4)
                *reinterpret_cast<float4*>(&part[warp][8 * c + j]) = make_float4(a[j], a[j + 1], a[j + 2], a[j + 3]);
        }
        __syncthreads();
        if (threadIdx.x < 128) {  // one column each: its maximum over the warps, its scale
            float t = part[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < 8; ++w) t = fmaxf(t, part[w][threadIdx.x]);
            part[0][threadIdx.x] = block_factor(t);
            const int n = k0 + static_cast<int>(threadIdx.x);
            if (n < p.K) p.SF[n * p.sf_pitch + blockIdx.y] = block_scale(t);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = part[0][8 * c + j];
    } else {
        float t = a[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) t = fmaxf(t, a[j]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, o));
        if (lane == 0) part[0][warp] = t;
        __syncthreads();
        t = part[0][0];
#pragma unroll
        for (int w = 1; w < 8; ++w) t = fmaxf(t, part[0][w]);
        if (threadIdx.x == 0)
            p.SF[LAYOUT == FP8_TILES ? blockIdx.y * p.sf_pitch + blockIdx.x : blockIdx.x * p.sf_pitch + blockIdx.y] = block_scale(t);
        t = block_factor(t);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = t;
    }
    if constexpr (!kTransposed) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = m0 + h * 64 + 4 * g + i, k = k0 + 8 * c;
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = to_f32(x[h][i].v[j]) * a[j];
                if (m < p.M && k < p.K)
                    *reinterpret_cast<uint2*>(p.Q + m * p.pitch + k) =
                        make_uint2(codes4(v[0], v[1], v[2], v[3]), codes4(v[4], v[5], v[6], v[7]));
            }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = to_f32(x[h][i].v[j]) * a[j];
                codes[(8 * c + j) * 32 + ((16 * h + g) ^ (2 * c))] = codes4(v[0], v[1], v[2], v[3]);
            }
        __syncthreads();
        // 16 lanes write a column's 128 bytes, 8 bytes (two words, kept together by the even
        // swizzle) each
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = i * 16 + (threadIdx.x >> 4), w = 2 * (threadIdx.x & 15);
            const uint2 v = *reinterpret_cast<const uint2*>(&codes[n * 32 + (w ^ (2 * (n >> 3)))]);
            if (k0 + n < p.K && m0 + 4 * w < p.pitch) *reinterpret_cast<uint2*>(p.Q + (k0 + n) * p.pitch + m0 + 4 * w) = v;
        }
    }
}

template <class T, int U>
cudaError_t launch_rows_of(const RowsParams& p, int64_t warps, cudaStream_t stream) {
    const int64_t segs = (int64_t(p.K) + U * 256 - 1) / (U * 256);
    int64_t y = (warps + p.R - 1) / p.R;  // segments side by side until there are `warps` warps
    y = y < segs ? y : segs;
    const int64_t x = (p.R + kThreads / 32 - 1) / (kThreads / 32);
    return launch_pdl(rows_kernel<T, U>, dim3(static_cast<unsigned>(x), static_cast<unsigned>(y < 65535 ? y : 65535)), dim3(kThreads), 0,
                      stream, p);
}

template <class T>
cudaError_t launch_rows(const RowsParams& p, int sms, cudaStream_t stream) {
    // As many pieces at a time as the row has, up to eight (128 bytes of 16-bit elements in
    // flight per lane), while that leaves eight warps per SM: few rows are cut finer.  1, 2, 4, 8
    // pieces (us): 4096 x 8192 26.7, 17.8, 13.9, 13.3; 1024 x 8192 7.1, 5.3, 4.1, 4.3; smaller
    // calls are within the launch's 3.7.
    const int64_t pieces = (int64_t(p.K) + 255) / 256, warps = int64_t(sms) * 8;
    auto fits = [&](int u) { return pieces >= u && p.R * ((pieces + u - 1) / u) >= warps; };
    if (fits(8)) return launch_rows_of<T, 8>(p, 4 * warps, stream);
    if (fits(4)) return launch_rows_of<T, 4>(p, 4 * warps, stream);
    if (fits(2)) return launch_rows_of<T, 2>(p, 4 * warps, stream);
    return launch_rows_of<T, 1>(p, 4 * warps, stream);
}

template <class T>
cudaError_t launch_tiles(const TileParams& p, int layout, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((p.K + 127) / 128), static_cast<unsigned>((p.M + 127) / 128));
    void (*kernel)(TileParams) = layout == FP8_COLS    ? tile_kernel<T, FP8_COLS>
                                 : layout == FP8_TILES ? tile_kernel<T, FP8_TILES>
                                                       : tile_kernel<T, FP8_TILES_T>;
    return launch_pdl(kernel, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace
}  // namespace tn

extern "C" gemm_status_t quantize_fp8(int64_t M, int64_t K, const void* X, int64_t ld, int dtype, int layout, int64_t R,
                                      const int32_t* index, int64_t index_div, void* Q, float* SF, cudaStream_t stream) {
    using namespace tn;
    constexpr int64_t kLimit = int64_t(1) << 31;
    if (M < 0 || M >= kLimit || K < 1 || K >= kLimit - kFp8Block || ld < K || ld >= kLimit || layout < FP8_ROWS || layout > FP8_TILES_T ||
        dtype < GEMM_DT_F32 || dtype > GEMM_DT_F16)
        return GEMM_ERR_INVALID_ARG;
    const bool rows = layout == FP8_ROWS, transposed = layout == FP8_COLS || layout == FP8_TILES_T;
    if (rows && (R < 0 || R >= kLimit || (index == nullptr && R != M) || index_div < 1 || index_div >= kLimit)) return GEMM_ERR_INVALID_ARG;
    if (!rows && index != nullptr) return GEMM_ERR_INVALID_ARG;
    // Tiles run down grid.y, whose limit is 65535.
    if (!rows && M > int64_t(65535) * 128) return GEMM_ERR_INVALID_ARG;
    const int64_t es = dtype == GEMM_DT_F32 ? 4 : 2;
    if (K % (transposed ? 8 : 16) != 0 || (ld * es) % 16 != 0) return GEMM_ERR_ALIGNMENT;
    if (rows ? R == 0 : M == 0) return GEMM_OK;
    if ((X == nullptr && M > 0) || Q == nullptr || SF == nullptr) return GEMM_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(Q) || !aligned_to(SF, 4) || !aligned_to(index, 4)) return GEMM_ERR_ALIGNMENT;
    const int64_t kb = (K + kFp8Block - 1) / kFp8Block, mb = (M + kFp8Block - 1) / kFp8Block, P = (M + 15) / 16 * 16;
    const uint64_t in = M > 0 ? (uint64_t(M - 1) * ld + K) * es : 0;
    const uint64_t out = rows ? uint64_t(R) * K : transposed ? uint64_t(K) * P : uint64_t(M) * K;
    const uint64_t sf = 4 * (rows ? uint64_t(R) * kb : layout == FP8_COLS ? uint64_t(K) * mb : uint64_t(kb) * mb);
    if (overlaps(Q, out, X, in) || overlaps(SF, sf, X, in) || overlaps(Q, out, SF, sf) ||
        (index != nullptr && (overlaps(Q, out, index, uint64_t(R) * 4) || overlaps(SF, sf, index, uint64_t(R) * 4))))
        return GEMM_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    const gemm_status_t st = device_info(&dev, &sms);
    if (st != GEMM_OK) return st;
    cudaError_t e;
    if (rows) {
        RowsParams p{};
        p.X = X;
        p.index = index;
        p.Q = static_cast<uint8_t*>(Q);
        p.SF = SF;
        p.M = M;
        p.ld = ld;
        p.R = R;
        p.K = static_cast<uint32_t>(K);
        p.blocks = static_cast<int>(kb);
        p.index_div = static_cast<int>(index_div);
        e = dtype == GEMM_DT_F32    ? launch_rows<float>(p, sms, stream)
            : dtype == GEMM_DT_BF16 ? launch_rows<__nv_bfloat16>(p, sms, stream)
                                    : launch_rows<__half>(p, sms, stream);
    } else {
        TileParams p{};
        p.X = X;
        p.Q = static_cast<uint8_t*>(Q);
        p.SF = SF;
        p.ld = ld;
        p.M = static_cast<int>(M);
        p.K = static_cast<int>(K);
        p.pitch = transposed ? P : K;
        p.sf_pitch = transposed ? mb : kb;
        e = dtype == GEMM_DT_F32    ? launch_tiles<float>(p, layout, stream)
            : dtype == GEMM_DT_BF16 ? launch_tiles<__nv_bfloat16>(p, layout, stream)
                                    : launch_tiles<__half>(p, layout, stream);
    }
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}
