// route_logits.cu -- experts of each token from given router logits: softmax or sigmoid
// scores, a selection-only bias, expert groups, TopK, weights.
//
//   s_e = softmax(r)_e or sigma(r_e),  key_e = s_e + b_e
//   score of group g (E / G neighbouring experts) = sum of its group_top largest keys
//   the topk_group groups of the largest score stay; I = TopK(key, K) inside them
//   w_e = s_e (/ sum_{j in I} s_j) * scale
// Ties go to the lower index.  A logit of -inf or NaN (or a key that becomes one) takes its
// expert out: it counts in no group score, comes after every other expert of the groups that
// stay, and has weight 0.  +inf counts as the largest finite number.
//
// The selection is the one of the real numbers s_e, not of their fp32 roundings.  Without a
// bias the logits themselves have the scores' order, so fp32 compares are exact (and a group
// judged by its best expert too).  Otherwise the keys are computed in fp32, and where two
// values that an output depends on come closer than the fp32 error bound below, the warp
// repeats its token in fp64 (about one token in 500 of normally distributed logits).
//
// One warp per token, expert e = 32 j + lane in register j.  Keys are kept as unsigned
// integers in the order of the floats, so that one redux.sync finds the best of a warp; a
// second one finds the lowest index that has it.  Bound by issue: a round costs about 4 E / 32
// instructions, the loads (4 E bytes a token) are a quarter of the time.
#include <algorithm>
#include <cfloat>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

// Order-preserving map of floats (no NaN) to unsigned integers above 0; 0 is free for "not a
// candidate".  -0 and +0 map alike.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const bf16* p) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
}

// NaN -> -inf (out), +inf -> the largest finite number
__device__ __forceinline__ float clean(float r) { return r == r ? fminf(r, FLT_MAX) : -INFINITY; }

// The token's logit e: the sum of the planes (in order) and the logit bias, if any.
template <typename T>
__device__ __forceinline__ float token_logit(const RouteLogitsLaunch& a, long long token, int e) {
    const T* p = reinterpret_cast<const T*>(a.logits) + token * a.row_stride + e;
    float r = load_logit(p);
    for (int q = 1; q < a.planes; ++q) r += load_logit(p + q * a.plane_stride);
    if (a.logit_bias) r += __ldg(a.logit_bias + e);
    return clean(r);
}

// The bound on the difference of two fp32 keys (or group scores) below which their order is
// not certain.  With a bias: a sigmoid is off by at most 5e-7, a softmax by 2e-6 (expf and the
// sum of 512 terms), the sum with the bias by 2^-24 of its size; a group score adds two of
// them.  Without: softmax sums, whose common denominator does not matter, by 1.2e-5 of their
// size for logits up to 100 below the largest (expf's argument is rounded); further
// down they are tiny or 0 and compare as equal.
__device__ __forceinline__ float uncertain(const RouteLogitsLaunch& a, float size) {
    if (a.select_bias == nullptr && a.score_mode == 0) return 3e-5f * fabsf(size);
    return (a.score_mode == 0 ? 1.2e-5f : 4e-6f) + 1e-6f * fabsf(size);
}

template <typename V>
__device__ __forceinline__ void keep_two(V& m1, V& m2, V v) {
    if (v > m1) { m2 = m1; m1 = v; }
    else if (v > m2) m2 = v;
}

// group score of the two best keys (-inf: none)
template <typename V>
__device__ __forceinline__ V group_score(V m1, V m2, int group_top) {
    return group_top == 2 && m2 > -INFINITY ? m1 + m2 : m1;
}

// The token's selection in fp64, by one warp: idx of slot k into lane k.  key: E doubles of
// this warp's shared memory.
template <typename T>
__device__ __noinline__ int select_fp64(const RouteLogitsLaunch& a, long long token, double* key,
                                        int lane) {
    const int E = a.E, S = E / a.n_group;
    double m = -INFINITY, z = 0.;
    if (a.score_mode == 0) {
        for (int e = lane; e < E; e += 32) m = fmax(m, static_cast<double>(token_logit<T>(a, token, e)));
        for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kAll, m, o));
        for (int e = lane; e < E; e += 32) {
            const double r = token_logit<T>(a, token, e);
            if (r > -INFINITY) z += exp(r - m);
        }
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
    }
    auto score = [&](double r) { return a.score_mode == 0 ? exp(r - m) / z : 1. / (1. + exp(-r)); };
    // without a bias the logits order the experts, also where scores underflow
    for (int e = lane; e < E; e += 32) {
        double k = token_logit<T>(a, token, e);
        if (a.select_bias && k > -INFINITY) {
            k = score(k) + static_cast<double>(__ldg(a.select_bias + e));
            if (!(k > -INFINITY)) k = -INFINITY;
        }
        key[e] = k;
    }
    __syncwarp();
    unsigned allowed = kAll;
    if (a.topk_group < a.n_group) {
        double m1 = -INFINITY, m2 = -INFINITY;
        if (lane < a.n_group)
            for (int i = 0; i < S; ++i) {
                const double k = key[lane * S + i];
                keep_two(m1, m2, a.select_bias == nullptr && k > -INFINITY ? score(k) : k);
            }
        const double mine = group_score(m1, m2, a.group_top);
        int before = 0;  // groups ahead of this lane's
        for (int g = 0; g < a.n_group; ++g) {
            const double o = __shfl_sync(kAll, mine, g);
            if (o > mine || (o == mine && g < lane)) ++before;
        }
        allowed = __ballot_sync(kAll, lane < a.n_group && before < a.topk_group);
    }
    unsigned taken = 0;  // of this lane's experts, by register j = e / 32
    int mine_k = 0;
    for (int k = 0; k < a.K; ++k) {
        double bv = -INFINITY;
        int bi = 0x7fffffff;
        for (int e = lane; e < E; e += 32) {
            if ((taken >> (e >> 5)) & 1u || !((allowed >> (e / S)) & 1u)) continue;
            if (bi == 0x7fffffff || key[e] > bv) { bv = key[e]; bi = e; }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(kAll, bv, o);
            const int oi = __shfl_xor_sync(kAll, bi, o);
            if (oi != 0x7fffffff && (bi == 0x7fffffff || ov > bv || (ov == bv && oi < bi))) {
                bv = ov;
                bi = oi;
            }
        }
        if ((bi & 31) == lane) taken |= 1u << (bi >> 5);
        if (lane == k) mine_k = bi;
    }
    __syncwarp();
    return mine_k;
}

template <typename T, int NV>
__device__ __forceinline__ void route_token(const RouteLogitsLaunch& a, long long token, float* sm,
                                            int* hist, int lane) {
    const int E = a.E, K = a.K, G = a.n_group, S = E / G;
    const bool grouped = a.topk_group < G;
    const bool on_logits = a.select_bias == nullptr;  // the logits have the keys' order
    const bool group_sums = grouped && a.group_top == 2;
    float r[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = j * 32 + lane;
        r[j] = e < E ? token_logit<T>(a, token, e) : -INFINITY;
    }
    float m = -INFINITY, z = 1.f;
    if (a.score_mode == 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) m = fmaxf(m, r[j]);
        m = unordered(__reduce_max_sync(kAll, ordered(m)));
        if (m == -INFINITY) m = 0.f;  // every expert out: scores 0
        if (!on_logits || !a.renorm) {
            z = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) z += expf(r[j] - m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
            if (z == 0.f) z = 1.f;
        }
    }
    auto score = [&](float v) { return a.score_mode == 0 ? expf(v - m) / z : 1.f / (1.f + expf(-v)); };
    uint32_t key[NV];
    bool sure = true;
    const int lpg = 32 / a.group_lanes;  // lanes that share a group's keys
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = j * 32 + lane;
        key[j] = 0u;
        if (e < E) {
            float k = r[j], in_group = r[j];
            if (!on_logits) {
                k = r[j] > -INFINITY ? score(r[j]) + __ldg(a.select_bias + e) : -INFINITY;
                in_group = k = k > -INFINITY ? k : -INFINITY;
            } else if (group_sums) {
                in_group = r[j] > -INFINITY ? score(r[j]) : -INFINITY;
            }
            key[j] = ordered(k);
            if (grouped) sm[e + ((e * a.group_magic) >> 20) * lpg] = in_group;
        }
    }
    if (grouped) {
        __syncwarp();
        const int g = lane / lpg, sub = lane % lpg;
        float m1 = -INFINITY, m2 = -INFINITY;
        if (g < G)
            for (int i = sub; i < S; i += lpg) keep_two(m1, m2, sm[g * (S + lpg) + i]);
        for (int o = lpg >> 1; o > 0; o >>= 1) {
            const float o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
            keep_two(m1, m2, o1);
            keep_two(m1, m2, o2);
        }
        __syncwarp();
        uint32_t gs = g < G && sub == 0 ? ordered(group_score(m1, m2, a.group_top)) : 0u;
        unsigned allowed = 0;
        uint32_t best = 0;
        for (int i = 0; i < a.topk_group; ++i) {
            best = __reduce_max_sync(kAll, gs);
            const int who = __ffs(__ballot_sync(kAll, gs == best)) - 1;  // the lowest group
            allowed |= 1u << (who / lpg);
            if (lane == who) gs = 0u;
        }
        if (!on_logits || group_sums) {
            const float last = unordered(best), next = unordered(__reduce_max_sync(kAll, gs));
            if (next > -INFINITY && !(last - next > uncertain(a, last))) sure = false;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = j * 32 + lane;
            if (!((allowed >> ((e * a.group_magic) >> 20)) & 1u)) key[j] = 0u;
        }
    }
    int my_e = 0;
    float prev = INFINITY;
    for (int k = 0; k < K; ++k) {
        uint32_t b = 0u;
#pragma unroll
        for (int j = 0; j < NV; ++j) b = max(b, key[j]);
        b = __reduce_max_sync(kAll, b);
        int e = 0x7fffffff;
#pragma unroll
        for (int j = NV - 1; j >= 0; --j)
            if (key[j] == b) e = j * 32 + lane;
        e = __reduce_min_sync(kAll, static_cast<unsigned>(e));
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * 32 + lane == e) key[j] = 0u;
        if (lane == k) my_e = e;
        const float v = unordered(b);
        if (!on_logits && v > -INFINITY && !(prev - v > uncertain(a, v))) sure = false;
        prev = v;
    }
    if (!on_logits) {  // the best one left out
        uint32_t b = 0u;
#pragma unroll
        for (int j = 0; j < NV; ++j) b = max(b, key[j]);
        b = __reduce_max_sync(kAll, b);
        const float v = b ? unordered(b) : -INFINITY;
        if (v > -INFINITY && !(prev - v > uncertain(a, v))) sure = false;
    }
    if (!sure) my_e = select_fp64<T>(a, token, reinterpret_cast<double*>(sm), lane);
    // weights: the selected scores, in the lanes of their slots
    float s = 0.f, l = -INFINITY;
    if (lane < K) {
        l = token_logit<T>(a, token, my_e);
        if (a.select_bias && l > -INFINITY && !(score(l) + __ldg(a.select_bias + my_e) > -INFINITY))
            l = -INFINITY;
        s = l > -INFINITY ? score(l) : 0.f;
    }
    if (a.renorm) {
        float sum = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        if (sum < 1e-30f) {
            // scores that (nearly) underflow: the same ratios from differences of logits, in
            // which sigma(r) = e^r to fp32 accuracy this far down
            float top = l;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
            s = l > -INFINITY ? expf(l - top) : 0.f;
            sum = s;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        }
        s = sum > 0.f ? s / sum : 0.f;
    }
    if (lane < K) {
        a.topk_idx[token * K + lane] = my_e;
        a.topk_w[token * K + lane] = s * a.scale;
        if (a.counts) atomicAdd(hist + my_e, 1);
    }
}

template <typename T, int NV>
__global__ void __launch_bounds__(kThreads) route_logits_kernel(const __grid_constant__ RouteLogitsLaunch a, int warp_bytes) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int hist[512];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* sm = reinterpret_cast<float*>(smem + static_cast<size_t>(warp) * warp_bytes);
    for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    for (long long t = static_cast<long long>(blockIdx.x) * kWarps + warp; t < a.T;
         t += static_cast<long long>(gridDim.x) * kWarps)
        route_token<T, NV>(a, t, sm, hist, lane);
    __syncthreads();
    if (a.counts)
        for (int e = threadIdx.x; e < a.E; e += kThreads) {
            if (gridDim.x == 1) a.counts[e] = hist[e];
            else if (hist[e]) atomicAdd(a.counts + e, hist[e]);
        }
}

template <typename T>
cudaError_t launch_typed(const RouteLogitsLaunch& a, int grid, size_t warp_bytes, cudaStream_t s,
                         bool pdl) {
    const int nv = ceil_div(a.E, 32);
    const size_t smem = kWarps * warp_bytes;
    auto go = [&](auto kernel) {
        return launch_kernel(kernel, dim3(grid), dim3(kThreads), smem, s, pdl, a,
                             static_cast<int>(warp_bytes));
    };
    return nv <= 1   ? go(route_logits_kernel<T, 1>)
           : nv <= 2 ? go(route_logits_kernel<T, 2>)
           : nv <= 4 ? go(route_logits_kernel<T, 4>)
           : nv <= 8 ? go(route_logits_kernel<T, 8>)
                     : go(route_logits_kernel<T, 16>);
}

}  // namespace

cudaError_t launch_route_logits(const RouteLogitsLaunch& in, int num_sms, cudaStream_t s, bool pdl) {
    RouteLogitsLaunch a = in;
    // up to 4 tokens a warp in one CTA, which writes the counts itself; otherwise the CTAs'
    // counts are added to cleared ones
    const bool one = a.T <= 4 * kWarps;
    if (a.counts && !one) {
        const cudaError_t err = cudaMemsetAsync(a.counts, 0, sizeof(int32_t) * a.E, s);
        if (err != cudaSuccess) return err;
    }
    if (a.T == 0 && !a.counts) return cudaSuccess;
    const int S = a.E / a.n_group;
    a.group_lanes = 1;
    while (a.group_lanes < a.n_group) a.group_lanes *= 2;
    a.group_magic = ((1 << 20) + S - 1) / S;  // e / S = e * magic >> 20 for e < 512
    // a warp's keys by group (each group padded against bank conflicts), or its fp64 keys
    const size_t padded = sizeof(float) * (a.E + static_cast<size_t>(a.n_group) * (32 / a.group_lanes));
    size_t warp_bytes = 0;
    if (a.select_bias || (a.topk_group < a.n_group && a.group_top == 2))
        warp_bytes = sizeof(double) * a.E;
    if (a.topk_group < a.n_group && warp_bytes < padded) warp_bytes = padded;
    warp_bytes = (warp_bytes + 15) & ~static_cast<size_t>(15);
    const int grid = one ? 1 : static_cast<int>(std::min<long long>(ceil_div(a.T, kWarps), 4ll * num_sms));
    const cudaError_t err = a.is_bf16 ? launch_typed<bf16>(a, grid, warp_bytes, s, pdl)
                                      : launch_typed<float>(a, grid, warp_bytes, s, pdl);
    count_launches(1);
    return err;
}

}  // namespace moe
