// Router of the expert layers: scores, (grouped) top-k and weights of each token, and
// the weights' gradient.
//
// LPT lanes per token (a warp, or 8 or 16 lanes where there are many tokens); lane l of a
// token holds the logits of experts l * VPT .. l * VPT + VPT-1 in registers, as keys mapped to
// unsigned integers in their own order, of which it sorts the L largest.  A pick is the
// maximum over the lanes' largest keys, a ballot for the lowest lane that holds it, and a
// shift of that lane's list.  The picks' indices are found afterwards, all at once: the
// lowest lane first and the lowest index within it is the lowest index among equal keys.
// The kernel is bound by its instructions.  Per token of 256 fp32 logits, sigmoid, bias, top 8
// of 4 of 8 groups (32768 tokens): 1300 instructions and 45 us taking picks out of unsorted
// lists; 1130 with sorted lists and a warp per token (32.1 us in the present kernel); 763 and
// 29.5 us with 16 lanes per token, where the steps across lanes serve two tokens at once, and
// four blocks per SM (the schedulers issue in 71 % of the cycles; the 36 MB would take 5 us).
// Eight lanes need 555 but 128 registers (34 us); they are used up to 128 experts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "experts.h"
#include "ptx.cuh"

namespace tn {
namespace {

constexpr int kRouteWarps = 8;  // per block
constexpr unsigned kFull = 0xffffffffu;

struct RouteParams {
    const void* logits;
    const float* bias;
    float* weights;
    int32_t* ids;
    const float* dweights;  // gradient only
    void* dlogits;
    int64_t ld, ldd;
    int64_t T;
    int E, top_k, groups, top_groups, group_best;
    bool renormalize, vec, vecb, vecd;
    float scale;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(float v, __half& o) { o = __float2half_rn(v); }

// VPT elements of type T moved as vectors of up to 16 bytes.
template <class T, int VPT>
struct alignas(VPT * sizeof(T) < 16 ? VPT * sizeof(T) : 16) Vec {
    T v[VPT];
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// A logit as the router sees it: NaN is -inf (masked), and -0 becomes +0 so that the
// integer order of the keys agrees with the comparison of floats.
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.0f : neg_inf(); }

template <class T, int VPT>
__device__ __forceinline__ void load_row(const T* row, int e0, int E, bool vec, float (&x)[VPT]) {
    if (vec && e0 + VPT <= E) {
        const Vec<T, VPT> v = *reinterpret_cast<const Vec<T, VPT>*>(row + e0);
#pragma unroll
        for (int i = 0; i < VPT; ++i) x[i] = clean(to_f32(v.v[i]));
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) x[i] = e0 + i < E ? clean(to_f32(row[e0 + i])) : neg_inf();
    }
}

// The definition's own operations in its order (exp, add, correctly rounded reciprocal),
// so that keys near one another compare as the definition's do.
__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.0f + expf(-x)); }

// exp(x - m) for the row maximum m: 0 for a masked logit, 1 for the maximum itself (an
// infinite maximum shares the row among its equals).
__device__ __forceinline__ float exp_below(float x, float m) {
    return x == neg_inf() ? 0.0f : x == m ? 1.0f : expf(x - m);
}

// Floats to unsigned integers of the same order, and back; every float maps above 0, which
// marks what cannot be chosen (and comes back as NaN, cleaned to -inf).
__device__ __forceinline__ uint32_t ordered(float f) {
    const int i = __float_as_int(f);
    return static_cast<uint32_t>(i ^ ((i >> 31) | INT32_MIN));
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return u == 0u ? neg_inf() : __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}

// Over the LPT lanes of a token (LPT consecutive lanes of the warp).
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t group_top(uint32_t v) {
    if constexpr (LPT == 32) return __reduce_max_sync(kFull, v);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
// The lowest lane of the token where `yes` holds (some lane's must).
template <int LPT>
__device__ __forceinline__ int group_first(bool yes, int base) {
    const unsigned b = __ballot_sync(kFull, yes) >> base;
    return __ffs(LPT == 32 ? b : b & ((1u << (LPT & 31)) - 1u)) - 1;
}
__device__ __forceinline__ float warp_sum(float v) { return group_sum<32>(v); }
__device__ __forceinline__ float warp_max(float v) { return group_max<32>(v); }

// Batcher's odd-even merge sort of VPT (a power of two) keys, descending.
__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}
template <int LO, int N, int R, int VPT>
__device__ __forceinline__ void odd_even_merge(uint32_t (&k)[VPT]) {
    constexpr int STEP = R * 2;
    if constexpr (STEP < N) {
        odd_even_merge<LO, N, STEP>(k);
        odd_even_merge<LO + R, N, STEP>(k);
#pragma unroll
        for (int i = LO + R; i + R < LO + N; i += STEP) order2(k[i], k[i + R]);
    } else {
        order2(k[LO], k[LO + R]);
    }
}
template <int LO, int N, int VPT>
__device__ __forceinline__ void sort_descending(uint32_t (&k)[VPT]) {
    if constexpr (N > 1) {
        sort_descending<LO, N / 2>(k);
        sort_descending<LO + N / 2, N / 2>(k);
        odd_even_merge<LO, N, 1>(k);
    }
}

// The L largest of the VPT keys, descending, in list: whole sort where L is VPT, else blocks
// of L sorted and merged: the elementwise larger of one descending list and the other
// reversed are the L largest of both, as a bitonic sequence.
template <int VPT, int L>
__device__ __forceinline__ void largest(const uint32_t (&key)[VPT], uint32_t (&list)[L]) {
    static_assert(VPT % L == 0, "whole blocks");
#pragma unroll
    for (int i = 0; i < L; ++i) list[i] = key[i];
    sort_descending<0, L>(list);
#pragma unroll
    for (int b = L; b < VPT; b += L) {
        uint32_t next[L];
#pragma unroll
        for (int i = 0; i < L; ++i) next[i] = key[b + i];
        sort_descending<0, L>(next);
#pragma unroll
        for (int i = 0; i < L; ++i) list[i] = max(list[i], next[L - 1 - i]);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < L; ++i)
                if ((i & o) == 0) order2(list[i], list[i + o]);
    }
}

// The two largest of (a, b) and (c, d), each pair in descending order.
__device__ __forceinline__ void merge2(float& a, float& b, float c, float d) {
    const float lo = fminf(a, c);
    a = fmaxf(a, c);
    b = fmaxf(lo, fmaxf(b, d));
}

template <class T, int VPT, int LPT, bool SIGMOID>
__global__ void __launch_bounds__(kRouteWarps * 32, VPT == 16 && LPT == 16 ? 4 : 1) route_kernel(const RouteParams p) {
    constexpr int TPW = 32 / LPT;                  // tokens per warp
    constexpr int L = LPT < 32 && VPT > 8 ? 8 : VPT;  // fewer lanes than a warp: at most 8 picks
    constexpr int NV = VPT < 4 ? 1 : VPT / 4;      // 16-byte vectors of a lane's keys
    // The keys by lane, to find the picks' indices in; vector v of lane l at v ^ l, free of bank conflicts.
    __shared__ __align__(16) uint32_t table[kRouteWarps][32 * VPT];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, gl = lane & (LPT - 1), base = lane - gl;
    uint32_t* mine = table[threadIdx.x >> 5];
    auto slot = [&](int l, int i) { return l * VPT + (VPT < 4 ? i : 4 * ((i / 4) ^ (l & (NV - 1))) + i % 4); };
    const int e0 = gl * VPT;
    const bool with_bias = p.bias != nullptr;
    const bool need_total = !SIGMOID && (with_bias || !p.renormalize);  // of the keys, or of the weights
    const int size = p.E / p.groups, lanes = size / VPT;  // experts, lanes of a run
    const bool cut = p.groups > 1 && p.top_groups < p.groups;
    // runs of a power of two of whole lanes; others go through the table (LPT = 32 alone)
    const bool whole = LPT < 32 || (size % VPT == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 32);
    float bias[VPT];
    if (with_bias) load_row<float, VPT>(p.bias, e0, p.E, p.vecb, bias);

    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5)) * TPW;
    if (t0 >= p.T) return;
    const bool real = t0 + base / LPT < p.T;  // past the last token: its last, not written
    const int64_t t = real ? t0 + base / LPT : p.T - 1;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    float x[VPT];
    load_row<T, VPT>(row, e0, p.E, p.vec, x);

    float m = 0.0f, total = 1.0f;  // softmax: row maximum and sum of exp(x - m)
    if (!SIGMOID) {
        m = x[0];
#pragma unroll
        for (int i = 1; i < VPT; ++i) m = fmaxf(m, x[i]);
        m = group_max<LPT>(m);
        if (need_total) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) total += exp_below(x[i], m);
            total = group_sum<LPT>(total);
        }
    }
    if (with_bias) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const float s = SIGMOID ? sigmoid(x[i]) : __fdiv_rn(exp_below(x[i], m), total);
            // (fmaxf: a NaN sum is -inf too)
            x[i] = x[i] == neg_inf() ? x[i] : fmaxf(__fadd_rn(s, bias[i]), neg_inf());
        }
    }
    // what a run's score adds: the key, but the score itself in a router without a bias
    const bool scores = !with_bias && p.group_best == 2;
    auto g = [&](float v) {
        if (!scores || v == neg_inf()) return v;
        return SIGMOID ? sigmoid(v) : exp_below(v, m);
    };
    auto best_runs = [&](float a, float b) {  // of the runs' best two keys, one run per lane
        const float score = clean(p.group_best == 2 && b != neg_inf() ? __fadd_rn(a, b) : a);
        uint32_t run = gl < p.groups ? ordered(score) : 0u;
        unsigned kept = 0;  // one by one, the lower first among equals
        for (int j = 0; j < p.top_groups; ++j) {
            const int src = group_first<LPT>(run == group_top<LPT>(run), base);
            kept |= 1u << src;
            if (gl == src) run = 0u;
        }
        return kept;
    };
    uint32_t key[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) key[i] = ordered(x[i]);
    if (p.E < LPT * VPT) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (e0 + i >= p.E) key[i] = 0u;
    }
    if (LPT == 32 && cut && !whole) {
        float* v = reinterpret_cast<float*>(mine);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (e0 + i < p.E) v[e0 + i] = g(x[i]);
        __syncwarp();
        float a = neg_inf(), b = neg_inf();
        if (lane < p.groups)
            for (int i = 0; i < size; ++i) merge2(a, b, v[lane * size + i], neg_inf());
        __syncwarp();
        const unsigned kept = best_runs(a, b);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (!(kept >> min((e0 + i) / size, 31) & 1u)) key[i] = 0u;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) mine[slot(lane, i)] = key[i];
    uint32_t list[L];
    largest<VPT, L>(key, list);
    if (cut && whole) {
        float a = g(unordered(list[0])), b = L > 1 ? g(unordered(list[L > 1 ? 1 : 0])) : neg_inf();
        for (int o = lanes >> 1; o > 0; o >>= 1) {
            const float c = __shfl_xor_sync(kFull, a, o), d = __shfl_xor_sync(kFull, b, o);
            merge2(a, b, c, d);
        }
        const int src = base + min(gl, p.groups - 1) * lanes;
        a = __shfl_sync(kFull, a, src);
        b = __shfl_sync(kFull, b, src);
        const unsigned kept = best_runs(a, b);
        if (!(kept >> min(gl / lanes, 31) & 1u)) {
#pragma unroll
            for (int i = 0; i < L; ++i) list[i] = 0u;
        }
    }

    // picks: lane j keeps the j-th key, its lane and how many equal ones that lane gave before
    uint32_t my_key = 0, prev_key = 0;
    int my_src = 0, my_nth = 0, prev_src = -1, nth = 0;
    for (int j = 0; j < p.top_k; ++j) {
        const uint32_t top = group_top<LPT>(list[0]);
        const int src = group_first<LPT>(list[0] == top, base);
        nth = src == prev_src && top == prev_key ? nth + 1 : 0;
        prev_src = src, prev_key = top;
        if (gl == src) {
#pragma unroll
            for (int i = 0; i + 1 < L; ++i) list[i] = list[i + 1];
            list[L - 1] = 0u;
        }
        if (gl == j) my_key = top, my_src = src, my_nth = nth;
    }
    __syncwarp();
    int id = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (mine[slot(base + my_src, i)] == my_key && my_nth-- == 0) id = my_src * VPT + i;

    // weights of the picks: the chosen logits are read again
    float s = 0.0f;
    const float v = gl < p.top_k ? clean(to_f32(row[id])) : neg_inf();
    if (SIGMOID) {
        if (gl < p.top_k) s = sigmoid(v);
    } else if (p.renormalize) {
        // shares of the chosen alone, below their own maximum (the gradient's way too): the row's
        // may be of an expert that the bias or the runs passed over, far above all of them
        s = exp_below(v, with_bias || cut ? group_max<LPT>(v) : m);
    } else {
        s = total > 0.0f ? exp_below(v, m) / total : 0.0f;
    }
    float w = s * p.scale;
    if (p.renormalize) {
        const float sum = group_sum<LPT>(s);
        w = sum > 0.0f ? p.scale * (s / sum) : 0.0f;
    }
    if (real && gl < p.top_k) {
        p.weights[t * p.top_k + gl] = w;
        p.ids[t * p.top_k + gl] = id;
    }
}

// Gradient: lane j holds pick j.  Renormalised weights depend on the chosen logits
// alone (for the softmax too: s_j / S = e_j / sum of the chosen e), so only those are
// read, and every other element of the row is 0; a softmax without it needs the row.
// 16391 tokens x 128 experts, bf16, 4 picks: with the routing itself 9.6 us, two launches
// whose 9 MB would take 1.4.
template <class T, int VPT, bool SIGMOID>
__global__ void __launch_bounds__(kRouteWarps * 32) route_grad_kernel(const RouteParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    T* out = static_cast<T*>(p.dlogits) + t * p.ldd;
    const int e0 = lane * VPT;

    int id = -1;
    float g = 0.0f, v = neg_inf();
    if (lane < p.top_k) {
        id = p.ids[t * p.top_k + lane];
        g = p.dweights[t * p.top_k + lane];
        if (id < 0 || id >= p.E) id = -1;
        if (id >= 0) v = clean(to_f32(row[id]));
    }
    float fill[VPT];  // the row where nothing was chosen
#pragma unroll
    for (int i = 0; i < VPT; ++i) fill[i] = 0.0f;
    float dx = 0.0f;
    if (SIGMOID) {
        // a masked logit has score 0 and gradient 0; 1 - s = sigmoid(-x) does not cancel
        const float s = id >= 0 ? sigmoid(v) : 0.0f;
        float share = s;
        float diff = g;
        if (p.renormalize) {
            const float sum = warp_sum(s);
            share = sum > 0.0f ? s / sum : 0.0f;
            diff = g - warp_sum(id >= 0 ? g * share : 0.0f);
        }
        dx = id >= 0 ? p.scale * share * diff * sigmoid(-v) : 0.0f;
    } else if (p.renormalize) {
        const float e = exp_below(v, warp_max(v));
        const float sum = warp_sum(e);
        const float share = sum > 0.0f ? e / sum : 0.0f;
        const float dot = warp_sum(id >= 0 ? g * share : 0.0f);
        dx = id >= 0 ? p.scale * share * (g - dot) : 0.0f;
    } else {
        float x[VPT];
        load_row<T, VPT>(row, e0, p.E, p.vec, x);
        float m = x[0];
#pragma unroll
        for (int i = 1; i < VPT; ++i) m = fmaxf(m, x[i]);
        m = warp_max(m);
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            fill[i] = exp_below(x[i], m);
            total += fill[i];
        }
        total = warp_sum(total);
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
        const float s = id >= 0 ? exp_below(v, m) * inv : 0.0f;
        const float dot = warp_sum(id >= 0 ? p.scale * g * s : 0.0f);
        dx = s * (p.scale * g - dot);
#pragma unroll
        for (int i = 0; i < VPT; ++i) fill[i] = -(fill[i] * inv) * dot;
    }
    if (p.vecd && e0 + VPT <= p.E) {
        Vec<T, VPT> o;
#pragma unroll
        for (int i = 0; i < VPT; ++i) from_f32(fill[i], o.v[i]);
        *reinterpret_cast<Vec<T, VPT>*>(out + e0) = o;
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (e0 + i < p.E) from_f32(fill[i], out[e0 + i]);
    }
    __syncwarp();  // the row's own elements before the picks'
    if (id >= 0) from_f32(dx, out[id]);
}

template <class T, int VPT>
RouteParams with_vectors(RouteParams q) {
    constexpr uintptr_t kAlign = alignof(Vec<T, VPT>);
    auto fits = [](const void* base, int64_t ld) {
        return reinterpret_cast<uintptr_t>(base) % kAlign == 0 && (ld * static_cast<int64_t>(sizeof(T))) % kAlign == 0;
    };
    q.vec = fits(q.logits, q.ld);
    q.vecb = q.bias != nullptr && reinterpret_cast<uintptr_t>(q.bias) % alignof(Vec<float, VPT>) == 0;
    q.vecd = q.dlogits != nullptr && fits(q.dlogits, q.ldd);
    return q;
}

template <class T, int VPT, int LPT>
cudaError_t launch_route(const RouteParams& p, int scoring, cudaStream_t stream) {
    constexpr int kTokens = kRouteWarps * (32 / LPT);
    const int64_t blocks = (p.T + kTokens - 1) / kTokens;
    return launch_pdl(scoring == ROUTE_SIGMOID ? route_kernel<T, VPT, LPT, true> : route_kernel<T, VPT, LPT, false>,
                      dim3(static_cast<unsigned>(blocks)), dim3(kRouteWarps * 32), 0, stream, with_vectors<T, VPT>(p));
}

template <class T, int VPT>
cudaError_t launch_grad(const RouteParams& p, int scoring, cudaStream_t stream) {
    const int64_t blocks = (p.T + kRouteWarps - 1) / kRouteWarps;
    return launch_pdl(scoring == ROUTE_SIGMOID ? route_grad_kernel<T, VPT, true> : route_grad_kernel<T, VPT, false>,
                      dim3(static_cast<unsigned>(blocks)), dim3(kRouteWarps * 32), 0, stream, with_vectors<T, VPT>(p));
}

template <class T>
cudaError_t launch_width(const RouteParams& p, int scoring, bool grad, int sms, cudaStream_t stream) {
    if (grad) {
        // elements per lane: the smallest power of two whose warp holds the row
        if (p.E <= 32) return launch_grad<T, 1>(p, scoring, stream);
        if (p.E <= 64) return launch_grad<T, 2>(p, scoring, stream);
        if (p.E <= 128) return launch_grad<T, 4>(p, scoring, stream);
        if (p.E <= 256) return launch_grad<T, 8>(p, scoring, stream);
        if (p.E <= 512) return launch_grad<T, 16>(p, scoring, stream);
        return launch_grad<T, 32>(p, scoring, stream);
    }
    // 8 or 16 lanes per token where the picks fit a lane's list and the runs are whole lanes, and
    // where there are tokens enough: with up to 64 experts for every scheduler, with more for
    // several rounds of them (a token's own time is longer on fewer lanes).  A warp, 8 or 16
    // lanes per token (us): 64 experts, 4096 tokens 4.4, 4.4, 16384 tokens 9.6, 6.9; 128 experts,
    // 8192 tokens 6.8, 8.5, 12288 tokens 9.3, 9.2, 32768 tokens 20.3, 14.2; 256 experts in 8
    // groups, 8192 tokens 10.0, 10.7, 14336 tokens 15.5, 14.9, 32768 tokens 32.1, 29.5.
    auto narrow = [&](int vpt) {
        const int size = p.E / p.groups, lanes = size / vpt;
        const bool whole = p.groups == 1 || p.top_groups == p.groups || (size % vpt == 0 && (lanes & (lanes - 1)) == 0);
        return p.top_k <= 8 && whole && p.T >= static_cast<int64_t>(sms) * (p.E <= 64 ? 16 : 80);
    };
    if (p.E <= 32) return narrow(4) ? launch_route<T, 4, 8>(p, scoring, stream) : launch_route<T, 1, 32>(p, scoring, stream);
    if (p.E <= 64) return narrow(8) ? launch_route<T, 8, 8>(p, scoring, stream) : launch_route<T, 2, 32>(p, scoring, stream);
    if (p.E <= 128) return narrow(16) ? launch_route<T, 16, 8>(p, scoring, stream) : launch_route<T, 4, 32>(p, scoring, stream);
    if (p.E <= 256) return narrow(16) ? launch_route<T, 16, 16>(p, scoring, stream) : launch_route<T, 8, 32>(p, scoring, stream);
    if (p.E <= 512) return launch_route<T, 16, 32>(p, scoring, stream);
    return launch_route<T, 32, 32>(p, scoring, stream);
}

gemm_status_t launch(const RouteParams& p, int dtype, int scoring, bool grad, int sms, cudaStream_t stream) {
    const cudaError_t e = dtype == GEMM_DT_F32    ? launch_width<float>(p, scoring, grad, sms, stream)
                          : dtype == GEMM_DT_BF16 ? launch_width<__nv_bfloat16>(p, scoring, grad, sms, stream)
                                                  : launch_width<__half>(p, scoring, grad, sms, stream);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

int elem_size(int dtype) { return dtype == GEMM_DT_F32 ? 4 : 2; }

bool route_sizes_ok(int64_t T, int64_t E, int64_t top_k, int64_t ld, int dtype, int scoring) {
    return T >= 0 && T < (int64_t(1) << 31) && E >= 1 && E <= kMaxExperts && top_k >= 1 && top_k <= 32 && top_k <= E &&
           ld >= E && ld < (int64_t(1) << 31) && dtype >= GEMM_DT_F32 && dtype <= GEMM_DT_F16 &&
           (scoring == ROUTE_SIGMOID || scoring == ROUTE_SOFTMAX);
}

}  // namespace
}  // namespace tn

extern "C" {

gemm_status_t expert_route(int64_t T, int64_t E, int64_t top_k, const void* logits, int64_t ld, int dtype,
                           const float* bias, float* weights, int32_t* ids, int scoring, int64_t groups,
                           int64_t top_groups, int group_best, int renormalize, float scale, cudaStream_t stream) {
    using namespace tn;
    if (!route_sizes_ok(T, E, top_k, ld, dtype, scoring)) return GEMM_ERR_INVALID_ARG;
    if (groups < 1 || groups > 32 || E % groups != 0 || top_groups < 1 || top_groups > groups ||
        (group_best != 1 && group_best != 2) || top_k > top_groups * (E / groups))
        return GEMM_ERR_INVALID_ARG;
    if (T == 0) return GEMM_OK;
    if (logits == nullptr || weights == nullptr || ids == nullptr) return GEMM_ERR_INVALID_ARG;
    const int es = elem_size(dtype);
    if (!aligned_to(logits, es) || !aligned_to(bias, 4) || !aligned_to(weights, 4) || !aligned_to(ids, 4))
        return GEMM_ERR_ALIGNMENT;
    const uint64_t in = (uint64_t(T - 1) * ld + E) * es, outb = uint64_t(T) * top_k * 4;
    if (overlaps(weights, outb, logits, in) || overlaps(ids, outb, logits, in) || overlaps(weights, outb, ids, outb) ||
        (bias != nullptr && (overlaps(weights, outb, bias, E * 4) || overlaps(ids, outb, bias, E * 4))))
        return GEMM_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    const gemm_status_t st = device_info(&dev, &sms);
    if (st != GEMM_OK) return st;
    RouteParams p{};
    p.logits = logits;
    p.bias = bias;
    p.weights = weights;
    p.ids = ids;
    p.ld = ld;
    p.T = T;
    p.E = static_cast<int>(E);
    p.top_k = static_cast<int>(top_k);
    p.groups = static_cast<int>(groups);
    p.top_groups = static_cast<int>(top_groups);
    p.group_best = group_best;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    return launch(p, dtype, scoring, false, sms, stream);
}

gemm_status_t expert_route_grad(int64_t T, int64_t E, int64_t top_k, const void* logits, int64_t ld, int dtype,
                                const int32_t* ids, const float* dweights, void* dlogits, int64_t ldd, int scoring,
                                int renormalize, float scale, cudaStream_t stream) {
    using namespace tn;
    if (!route_sizes_ok(T, E, top_k, ld, dtype, scoring) || ldd < E || ldd >= (int64_t(1) << 31))
        return GEMM_ERR_INVALID_ARG;
    if (T == 0) return GEMM_OK;
    if (logits == nullptr || ids == nullptr || dweights == nullptr || dlogits == nullptr) return GEMM_ERR_INVALID_ARG;
    const int es = elem_size(dtype);
    if (!aligned_to(logits, es) || !aligned_to(dlogits, es) || !aligned_to(ids, 4) || !aligned_to(dweights, 4))
        return GEMM_ERR_ALIGNMENT;
    const uint64_t in = (uint64_t(T - 1) * ld + E) * es, out = (uint64_t(T - 1) * ldd + E) * es;
    const uint64_t pairs = uint64_t(T) * top_k * 4;
    if (overlaps(dlogits, out, logits, in) || overlaps(dlogits, out, ids, pairs) || overlaps(dlogits, out, dweights, pairs))
        return GEMM_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    const gemm_status_t st = device_info(&dev, &sms);
    if (st != GEMM_OK) return st;
    RouteParams p{};
    p.logits = logits;
    p.ids = const_cast<int32_t*>(ids);
    p.dweights = dweights;
    p.dlogits = dlogits;
    p.ld = ld;
    p.ldd = ldd;
    p.T = T;
    p.E = static_cast<int>(E);
    p.top_k = static_cast<int>(top_k);
    p.groups = 1;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    return launch(p, dtype, scoring, true, sms, stream);
}

}  // extern "C"
