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
// values that an output depends on come closer than the fp32 error bound (`uncertain`), the
// warp decides in fp64: between groups from all keys, between experts from the few that are
// still in question.
//
// One warp per token, expert e = 32 j + lane in register j.  Keys are kept as unsigned
// integers in the order of the floats.  TopK in two steps: the K-th best of the 32 lanes' own
// maxima bounds the K-th best key from below; the keys that reach it (K to about 2 K of them)
// are gathered, one to a lane, and each lane counts the ones before its own.  Counting
// against values broadcast from shared memory is a short chain of independent compares;
// K rounds of warp-wide maxima over all registers were a chain of K times the latency and
// four instructions a round and register.  Groups of 32 experts are single registers, judged
// by warp-wide maxima; others go through shared memory.
//
// 16381 x 256 fp32 logits, K = 8, 3 of 8 groups by their best key: 20.7 us (17 MB, 2.6 us of memory
// traffic; 34.8 with K rounds), bound by instruction issue (800 instructions a token, 2.3 of 4
// slots used).  4096 x 512, K = 10, 5 of 16 groups by two keys, bias: 20.2 us (58.9 with K rounds and
// every doubtful token decided in fp64 from all of its keys), a chain of latencies (1.1 of 4 slots,
// 39% of the warps).  One token 4.9 us.  Groups of 20, 32, 40 and 64 experts and none, the same rules on
// other logits: 16381 x 240 or 256: 26.6, 20.5, 26.0, 24.7, 18.4 us; 4096 x 480 or 512: 19.0, 18.6,
// 19.4, 19.8, 15.6.
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
    const int b = __float_as_int(v + 0.f);
    return static_cast<uint32_t>(b ^ ((b >> 31) | static_cast<int>(0x80000000u)));
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const bf16* p) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
}

// NaN -> -inf (out), +inf -> the largest finite number
__device__ __forceinline__ float clean(float r) { return fminf(fmaxf(r, -INFINITY), FLT_MAX); }

// The token's logit e: the sum of the planes (in order) and the logit bias, if any.
template <typename T>
__device__ __forceinline__ float token_logit(const RouteLogitsLaunch& a, long long token, int e) {
    const T* p = reinterpret_cast<const T*>(a.logits) + token * a.row_stride + e;
    float r = load_logit(p);
    for (int q = 1; q < a.planes; ++q) r += load_logit(p + q * a.plane_stride);
    if (a.logit_bias) r += __ldg(a.logit_bias + e);
    return clean(r);
}

// 1 / v to 1 ulp (0 for +inf)
__device__ __forceinline__ float quick_reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// What two fp32 keys (size: of the larger) have to differ by for their order to be certain, with a
// bias: a sigmoid is off by at most 5e-7 (its exponential's relative error counts
// s (1 - s) <= 1/4 times, and |r| s (1 - s) <= 0.23; a reciprocal by 2 ulp), a softmax by 3e-6 (the
// same exponential and a sum of 512 terms), the sum with the bias by 2^-24 of its size.
__device__ __forceinline__ float uncertain(const RouteLogitsLaunch& a, float size) {
    return (a.score_mode == 0 ? 6e-6f : 1.3e-6f) + 2.5e-7f * fabsf(size);
}

// How far what a group is judged by may be off, size: the sum of its (at most two) keys'
// magnitudes; their own sum may be far smaller, with biases of either sign, and its error is not.
// With a bias as two keys differ above (2^-24 of size for the keys and as much for the sum).  Without
// one only sums of scores are not exact (their common denominator does not matter): a term is off by
// (|r - max| + 4) 2^-23 of its size, 1.5e-5 for logits down to 100 below the largest, and where it
// is below the smallest normal number, by that.
__device__ __forceinline__ float group_error(const RouteLogitsLaunch& a, float size) {
    return a.select_bias ? uncertain(a, size) : 1.5e-5f * size + 2.5e-38f;
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

// The scores in fp64 (m, z: largest logit and sum of exponentials; softmax only).
struct Exact {
    double m, z;
    __device__ __forceinline__ double score(const RouteLogitsLaunch& a, float r) const {
        return a.score_mode == 0 ? exp(static_cast<double>(r) - m) / z
                                 : 1. / (1. + exp(-static_cast<double>(r)));
    }
    // score + bias; -inf for an expert that is out
    __device__ __forceinline__ double key(const RouteLogitsLaunch& a, float r, int e) const {
        if (!(r > -INFINITY)) return -INFINITY;
        double k = score(a, r);
        if (a.select_bias) k += static_cast<double>(__ldg(a.select_bias + e));
        return k > -INFINITY ? k : -INFINITY;
    }
    // the same order; without a bias the logits have it, also where scores underflow
    __device__ __forceinline__ double order(const RouteLogitsLaunch& a, float r, int e) const {
        return a.select_bias ? key(a, r, e) : static_cast<double>(r);
    }
};

template <typename T>
__device__ __noinline__ Exact exact_scores(const RouteLogitsLaunch& a, long long token, int lane) {
    Exact x{-INFINITY, 0.};
    if (a.score_mode == 0) {
        for (int e = lane; e < a.E; e += 32) x.m = fmax(x.m, static_cast<double>(token_logit<T>(a, token, e)));
        for (int o = 16; o > 0; o >>= 1) x.m = fmax(x.m, __shfl_xor_sync(kAll, x.m, o));
#pragma unroll 4
        for (int e = lane; e < a.E; e += 32) {
            const float r = token_logit<T>(a, token, e);
            if (r > -INFINITY) x.z += exp(static_cast<double>(r) - x.m);
        }
        for (int o = 16; o > 0; o >>= 1) x.z += __shfl_xor_sync(kAll, x.z, o);
    }
    return x;
}

// The `want` best of the groups in `near` (a bit each), by their scores in fp64; the warp goes
// through one group at a time, an expert to a lane.
template <typename T>
__device__ __noinline__ unsigned exact_groups(const RouteLogitsLaunch& a, long long token, unsigned near,
                                              int want, int lane) {
    const int S = a.group_size;
    const Exact x = exact_scores<T>(a, token, lane);
    double mine = -INFINITY;  // lane g: the score of group g
    for (unsigned left = near; left; left &= left - 1) {
        const int g = __ffs(left) - 1;
        double m1 = -INFINITY, m2 = -INFINITY;
        for (int i = lane; i < S; i += 32) {
            const int e = g * S + i;
            keep_two(m1, m2, x.key(a, token_logit<T>(a, token, e), e));
        }
        for (int o = 16; o > 0; o >>= 1) {
            const double o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
            keep_two(m1, m2, o1);
            keep_two(m1, m2, o2);
        }
        if (lane == g) mine = group_score(m1, m2, a.group_top);
    }
    int before = 0;  // near groups ahead of this lane's
    for (unsigned left = near; left; left &= left - 1) {
        const int g = __ffs(left) - 1;
        const double o = __shfl_sync(kAll, mine, g);
        if (o > mine || (o == mine && g < lane)) ++before;
    }
    return __ballot_sync(kAll, ((near >> lane) & 1u) && before < want);
}

// TopK in fp64 over every expert of the allowed groups: the expert of slot k into lane k.
template <typename T>
__device__ __noinline__ int exact_topk(const RouteLogitsLaunch& a, long long token, double* key,
                                       unsigned allowed, int lane) {
    const int E = a.E, S = a.group_size;
    const Exact x = exact_scores<T>(a, token, lane);
    for (int e = lane; e < E; e += 32) key[e] = x.order(a, token_logit<T>(a, token, e), e);
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

// The K first of the lanes' candidates (e: expert; live: has one), by fp64 key:
// the expert of slot k into lane k.
template <typename T>
__device__ __noinline__ int exact_order(const RouteLogitsLaunch& a, long long token, int e, bool live,
                                        int lane) {
    const Exact x = exact_scores<T>(a, token, lane);
    const double k = live ? x.key(a, token_logit<T>(a, token, e), e) : -INFINITY;
    int rank = 0;
#pragma unroll 4
    for (int l = 0; l < 32; ++l) {
        const double o = __shfl_sync(kAll, k, l);
        const int oe = __shfl_sync(kAll, live ? e : 0x7fffffff, l);
        if (oe != 0x7fffffff && (o > k || (o == k && oe < e))) ++rank;
    }
    int mine = 0;
    for (int s = 0; s < a.K; ++s) {
        const int who = __ffs(__ballot_sync(kAll, live && rank == s)) - 1;
        const int v = __shfl_sync(kAll, e, who);
        if (lane == s) mine = v;
    }
    return mine;
}

// A key and the index that decides between equal ones (the lower first), as one number in the
// order of the selection.
__device__ __forceinline__ uint64_t with_index(uint32_t key, uint32_t index) {
    return static_cast<uint64_t>(key) << 32 | (0xffffu - index);
}
__device__ __forceinline__ uint32_t index_of(uint64_t v) { return 0xffffu - static_cast<uint32_t>(v); }

// How many of the n values in buf (shared memory, 16-byte aligned, followed by 0 where n is odd)
// are larger than v.
__device__ __forceinline__ int count_larger(const uint64_t* buf, int n, uint64_t v) {
    int rank = 0;
    for (int q = 0; q < n; q += 2) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(buf + q);
        rank += (o.x > v) + (o.y > v);
    }
    return rank;
}

// What a group is judged by, from its two best keys (0: none), and the sum of their magnitudes (0
// where the best one is infinite: nothing is uncertain then).
struct Judged {
    uint32_t value;
    float size;
};
__device__ __forceinline__ Judged judged(const RouteLogitsLaunch& a, uint32_t m1, uint32_t m2) {
    const float k1 = unordered(m1), k2 = m2 ? unordered(m2) : -INFINITY;
    const bool finite = fabsf(k1) < INFINITY;
    if (a.group_top == 1) return {m1, finite ? fabsf(k1) : 0.f};
    return {ordered(group_score(k1, k2, 2)),
            finite ? fabsf(k1) + (k2 > -INFINITY ? fabsf(k2) : 0.f) : 0.f};
}

// Groups of 32 experts are one register of the warp each: lane g gets what group g is judged by,
// from one or two warp-wide maxima a group.
template <int NV>
__device__ __forceinline__ Judged groups_in_registers(const RouteLogitsLaunch& a,
                                                      const uint32_t (&key)[NV], int lane) {
    uint32_t m1 = 0u, m2 = 0u;
#pragma unroll
    for (int g = 0; g < NV; ++g) {
        const uint32_t w = __reduce_max_sync(kAll, key[g]);
        if (lane == g) m1 = w;
    }
    if (a.group_top == 2) {
#pragma unroll
        for (int g = 0; g < NV; ++g) {  // the best without one lane that holds the best
            const uint32_t w1 = __shfl_sync(kAll, m1, g);
            const int who = __ffs(__ballot_sync(kAll, key[g] == w1)) - 1;
            const uint32_t w = __reduce_max_sync(kAll, lane == who ? 0u : key[g]);
            if (lane == g) m2 = w;
        }
    }
    return judged(a, m1, m2);
}

// The same for groups of any size, whose keys are in sm, each group padded: group_lpg lanes (a
// power of two) look through a group, and all of them get its value.
__device__ __forceinline__ Judged groups_in_memory(const RouteLogitsLaunch& a, const uint32_t* sm, int lane) {
    const int S = a.group_size, lpg = a.group_lpg;
    const int g = lane >> a.group_shift, sub = lane & (lpg - 1);
    uint32_t m1 = 0u, m2 = 0u;
    if (g < a.n_group) {
        const uint32_t* k = sm + g * (S + a.group_pad);
        for (int i = sub; i < S; i += lpg) keep_two(m1, m2, k[i]);
    }
    for (int o = lpg >> 1; o > 0; o >>= 1) {
        const uint32_t o1 = __shfl_xor_sync(kAll, m1, o), o2 = __shfl_xor_sync(kAll, m2, o);
        m2 = max(min(m1, o1), max(m2, o2));
        m1 = max(m1, o1);
    }
    return judged(a, m1, m2);
}

// The groups that stay (a bit each): j is what group g is judged by, in the lanes that speak for
// one.  *near: the groups on either side of the border whose scores are not certain to be on
// theirs (0: none).
__device__ __forceinline__ unsigned pick_groups(const RouteLogitsLaunch& a, Judged j, int g, bool speaks,
                                                bool exact, unsigned* near, int lane) {
    unsigned allowed = 0;
    uint32_t left = speaks ? j.value : 0u;
    for (int i = 0; i < a.topk_group; ++i) {
        // the best one left; equal ones: the lowest lane, which speaks for the lowest group
        const unsigned who = __ballot_sync(kAll, left == __reduce_max_sync(kAll, left));
        const int first = __ffs(who) - 1;
        allowed |= 1u << (first >> a.speaker_shift);
        if (lane == first) left = 0u;
    }
    const bool stays = speaks && left == 0u;
    *near = 0;
    if (!exact) {
        // the score lies between lo and hi
        const float v = unordered(j.value), err = group_error(a, j.size);
        const bool known = err < INFINITY;
        const float lo = known ? v - err : -INFINITY, hi = known ? v + err : INFINITY;
        const float last = unordered(__reduce_min_sync(kAll, stays ? ordered(lo) : 0xffffffffu));
        const float after = unordered(__reduce_max_sync(kAll, speaks && !stays ? ordered(hi) : 0u));
        if (after > -INFINITY && !(last > after))
            *near = __reduce_or_sync(
                kAll, speaks && (stays ? !(lo > after) : hi > -INFINITY && !(last > hi)) ? 1u << g : 0u);
    }
    return allowed;
}

// Renormalised weights of the slots' logits l by their differences: those of a softmax, and of
// sigmoids that are all below 4e-8, where sigma(r) = e^r to fp32 accuracy.  However small the scores
// are, the ratios keep their digits.
__device__ __forceinline__ float weight_by_difference(float l) {
    const float best = unordered(__reduce_max_sync(kAll, ordered(l)));
    const float s = l > -INFINITY ? expf(l - best) : 0.f;
    float sum = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    return sum > 0.f ? s / sum : 0.f;
}

// SUMS: the logits come in planes or with a bias.  The code is kept short (the rare paths are
// calls): a launch of few tokens is bound by fetching it.
template <typename T, int NV, bool SIGMOID, bool SUMS>
__device__ __forceinline__ void route_token(const RouteLogitsLaunch& a, long long token,
                                            const float (&bias)[NV], uint32_t* sm, int* hist,
                                            int lane) {
    const int E = a.E, K = a.K;
    const bool grouped = a.topk_group < a.n_group;
    const bool on_logits = a.select_bias == nullptr;  // the logits have the keys' order
    const bool group_sums = grouped && a.group_top == 2;
    const T* row = reinterpret_cast<const T*>(a.logits) + token * a.row_stride + lane;
    float r[NV];
#pragma unroll
    // (past E: out, and behind every real expert that is)
    for (int j = 0; j < NV; ++j) r[j] = j * 32 + lane < E ? load_logit(row + j * 32) : -INFINITY;
    if (SUMS) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (j * 32 + lane >= E) continue;
            for (int q = 1; q < a.planes; ++q) r[j] += load_logit(row + j * 32 + q * a.plane_stride);
            if (a.logit_bias) r[j] += __ldg(a.logit_bias + j * 32 + lane);
        }
    }
    float m = 0.f, z = 1.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) r[j] = clean(r[j]);
    if (!SIGMOID) {
        m = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) m = fmaxf(m, r[j]);
        m = unordered(__reduce_max_sync(kAll, ordered(m)));
        if (m == -INFINITY) m = 0.f;  // every expert out: scores 0
        if (!on_logits || !a.renorm) {
            z = 0.f;
#pragma unroll
            for (int j = 0; j < NV; ++j) z += __expf(r[j] - m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
            if (z == 0.f) z = 1.f;
        }
    }
    uint32_t key[NV];
    if (on_logits && !group_sums) {
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = ordered(r[j]);
    } else {
        // scores for comparing (the weights below are computed with expf and divisions)
        const float inv_z = __fdividef(1.f, z);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float k = SIGMOID ? quick_reciprocal(1.f + __expf(-r[j])) : __expf(r[j] - m) * inv_z;
            k += bias[j];  // (0 without one)
            key[j] = ordered(r[j] > -INFINITY ? fmaxf(k, -INFINITY) : -INFINITY);
        }
    }
    unsigned allowed = kAll;
    if (grouped) {
        Judged gs;
        int g = lane;
        bool speaks = lane < a.n_group;
        if (a.whole_registers) {
            gs = groups_in_registers<NV>(a, key, lane);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int e = j * 32 + lane;
                if (e < E) sm[e + ((e * a.group_magic) >> 20) * a.group_pad] = key[j];
            }
            __syncwarp();
            gs = groups_in_memory(a, sm, lane);
            g = lane >> a.group_shift;
            speaks = g < a.n_group && (lane & (a.group_lpg - 1)) == 0;
        }
        unsigned near;
        allowed = pick_groups(a, gs, g, speaks, on_logits && !group_sums, &near, lane);
        if (near) {
            const unsigned sure = allowed & ~near;
            allowed = sure | exact_groups<T>(a, token, near, a.topk_group - __popc(sure), lane);
        }
        if (on_logits && group_sums) {
#pragma unroll
            for (int j = 0; j < NV; ++j) key[j] = ordered(r[j]);
        }
        if (a.whole_registers) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (!(allowed & (1u << j))) key[j] = 0u;
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int e = j * 32 + lane;  // (past E: 0, the group may not exist)
                if (e >= E || !((allowed >> ((e * a.group_magic) >> 20)) & 1u)) key[j] = 0u;
            }
        }
    }
    // A lower bound of the K-th best key: the K-th best of the lanes' maxima (0: fewer lanes than
    // K have a candidate, so every candidate counts).
    uint32_t top = 0u;
#pragma unroll
    for (int j = 0; j < NV; ++j) top = max(top, key[j]);
    __syncwarp();
    sm[lane] = top;
    __syncwarp();
    int above = 0;
#pragma unroll
    for (int q = 0; q < 32; q += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(sm + q);
        above += (o.x > top) + (o.y > top) + (o.z > top) + (o.w > top);
    }
    const uint32_t bound = __reduce_min_sync(kAll, above < K ? top : 0xffffffffu);
    // what may still come before an expert at the bound in real numbers
    uint32_t low = max(bound, 1u);
    if (!on_logits && bound) {
        const float v = unordered(bound);
        if (v > -INFINITY && v < INFINITY) low = ordered(v - uncertain(a, v));
    }
    // candidates to shared memory, lane by lane
    uint64_t* cand = reinterpret_cast<uint64_t*>(sm);
    int own = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) own += key[j] >= low;
    int at = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, at, o);
        if (lane >= o) at += v;
    }
    const int n = __shfl_sync(kAll, at, 31);
    int my_e = 0;
    float l = -INFINITY;  // the slot's logit
    if (n >= K && n <= 32) {
        at -= own;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (key[j] >= low) cand[at++] = with_index(key[j], j * 32 + lane);
        if (lane == 0) cand[n] = 0u;
        __syncwarp();
        const uint64_t mine = cand[lane];
        const int rank = lane < n ? count_larger(cand, n, mine) : 32;
        uint64_t* slot = cand + 34;  // K + 1 places
        if (lane == K) slot[K] = 0u;
        __syncwarp();
        if (rank <= K) slot[rank] = mine;
        __syncwarp();
        bool sure = true;
        if (lane < K) {
            const uint32_t k = static_cast<uint32_t>(slot[lane] >> 32);
            my_e = static_cast<int>(index_of(slot[lane]));
            if (on_logits) {
                l = unordered(k);
            } else {
                l = token_logit<T>(a, token, my_e);
                const uint32_t after = static_cast<uint32_t>(slot[lane + 1] >> 32);
                const float v = unordered(k), va = after ? unordered(after) : -INFINITY;
                sure = va == -INFINITY || v - va > uncertain(a, v);
            }
        }
        if (!__all_sync(kAll, sure)) {
            const int e = static_cast<int>(index_of(mine));
            my_e = exact_order<T>(a, token, e, lane < n && e < E, lane);
            if (lane < K) l = token_logit<T>(a, token, my_e);
        }
    } else {
        // many keys that (nearly) equal the bound
        my_e = exact_topk<T>(a, token, reinterpret_cast<double*>(sm), allowed, lane);
        if (lane < K) l = token_logit<T>(a, token, my_e);
    }
    // weights: the selected scores, in the lanes of their slots (an expert that is out: 0)
    if (lane < K && a.select_bias && !(__ldg(a.select_bias + my_e) > -INFINITY)) l = -INFINITY;
    float w = 0.f;
    if (!SIGMOID && a.renorm) {
        w = weight_by_difference(l);
    } else if (!SIGMOID) {
        if (l > -INFINITY) w = expf(l - m) / z;
    } else {
        const float e = expf(-fabsf(l));  // at most 1: no overflow, and subnormal scores survive
        if (l > -INFINITY) w = (l < 0.f ? e : 1.f) / (1.f + e);
        if (a.renorm) {
            float sum = w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            w = sum < 4e-8f ? weight_by_difference(l) : w / sum;
        }
    }
    if (lane < K) {
        a.topk_idx[token * K + lane] = my_e;
        a.topk_w[token * K + lane] = w * a.scale;
        if (a.counts) atomicAdd(hist + my_e, 1);
    }
}

template <typename T, int NV, bool SIGMOID, bool SUMS>
__global__ void __launch_bounds__(kThreads, 4)
route_logits_kernel(const __grid_constant__ RouteLogitsLaunch a, int warp_bytes) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int hist[512];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* sm = reinterpret_cast<uint32_t*>(smem + static_cast<size_t>(warp) * warp_bytes);
    for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    float bias[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        bias[j] = a.select_bias && j * 32 + lane < a.E ? __ldg(a.select_bias + j * 32 + lane) : 0.f;
    for (long long t = static_cast<long long>(blockIdx.x) * kWarps + warp; t < a.T;
         t += static_cast<long long>(gridDim.x) * kWarps)
        route_token<T, NV, SIGMOID, SUMS>(a, t, bias, sm, hist, lane);
    __syncthreads();
    if (a.counts)
        for (int e = threadIdx.x; e < a.E; e += kThreads) {
            if (gridDim.x == 1) a.counts[e] = hist[e];
            else if (hist[e]) atomicAdd(a.counts + e, hist[e]);
        }
}

template <typename T, bool SIGMOID, bool SUMS>
cudaError_t launch_typed(const RouteLogitsLaunch& a, int grid, size_t warp_bytes, cudaStream_t s,
                         bool pdl) {
    const int nv = ceil_div(a.E, 32);
    const size_t smem = kWarps * warp_bytes;
    auto go = [&](auto kernel) {
        return launch_kernel(kernel, dim3(grid), dim3(kThreads), smem, s, pdl, a,
                             static_cast<int>(warp_bytes));
    };
    return nv <= 1   ? go(route_logits_kernel<T, 1, SIGMOID, SUMS>)
           : nv <= 2 ? go(route_logits_kernel<T, 2, SIGMOID, SUMS>)
           : nv <= 4 ? go(route_logits_kernel<T, 4, SIGMOID, SUMS>)
           : nv <= 8 ? go(route_logits_kernel<T, 8, SIGMOID, SUMS>)
                     : go(route_logits_kernel<T, 16, SIGMOID, SUMS>);
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
    a.group_size = S;
    a.whole_registers = S == 32;
    a.group_magic = ((1 << 20) + S - 1) / S;  // e / S = e * magic >> 20 for e < 512
    a.group_shift = 5;
    while ((32 >> a.group_shift) < a.n_group) --a.group_shift;
    a.group_lpg = 1 << a.group_shift;
    a.speaker_shift = a.whole_registers ? 0 : a.group_shift;
    a.group_pad = a.group_lpg;  // keeps the lanes' reads off each other's banks
    // a warp's shared memory: the keys by group, each group padded; candidates and slots; the
    // fp64 keys of the rare paths
    size_t warp_bytes = std::max<size_t>(sizeof(uint64_t) * (34 + 18), sizeof(double) * a.E);
    if (a.topk_group < a.n_group)
        warp_bytes = std::max(warp_bytes, sizeof(uint32_t) * (a.E + static_cast<size_t>(a.n_group) * a.group_pad));
    warp_bytes = (warp_bytes + 15) & ~static_cast<size_t>(15);
    const int grid = one ? 1 : static_cast<int>(std::min<long long>(ceil_div(a.T, kWarps), 4ll * num_sms));
    // (bf16 logits are given ones: no planes, no bias)
    const bool sums = a.planes > 1 || a.logit_bias != nullptr, sigmoid = a.score_mode != 0;
    const cudaError_t err =
        a.is_bf16 ? (sigmoid ? launch_typed<bf16, true, false>(a, grid, warp_bytes, s, pdl)
                             : launch_typed<bf16, false, false>(a, grid, warp_bytes, s, pdl))
        : sums    ? (sigmoid ? launch_typed<float, true, true>(a, grid, warp_bytes, s, pdl)
                             : launch_typed<float, false, true>(a, grid, warp_bytes, s, pdl))
                  : (sigmoid ? launch_typed<float, true, false>(a, grid, warp_bytes, s, pdl)
                             : launch_typed<float, false, false>(a, grid, warp_bytes, s, pdl));
    count_launches(1);
    return err;
}

}  // namespace moe
