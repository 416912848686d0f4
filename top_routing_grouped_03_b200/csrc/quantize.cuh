// quantize.cuh -- the device side of quantize.cu: a row's scale and the rounding of its values
// (the formulas and the exactness of the rounding are explained there).
#pragma once

#include "common.cuh"

namespace moe {
namespace {

// 16 values as fp32
__device__ __forceinline__ void load_chunk(const bf16* p, float (&v)[16]) {
    const uint4* s = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 w = __ldg(s + h);
        v[8 * h] = bf16_lo(w.x); v[8 * h + 1] = bf16_hi(w.x);
        v[8 * h + 2] = bf16_lo(w.y); v[8 * h + 3] = bf16_hi(w.y);
        v[8 * h + 4] = bf16_lo(w.z); v[8 * h + 5] = bf16_hi(w.z);
        v[8 * h + 6] = bf16_lo(w.w); v[8 * h + 7] = bf16_hi(w.w);
    }
}
__device__ __forceinline__ void load_chunk(const float* p, float (&v)[16]) {
    const float4* s = reinterpret_cast<const float4*>(p);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float4 w = __ldcg(s + h);
        v[4 * h] = w.x; v[4 * h + 1] = w.y; v[4 * h + 2] = w.z; v[4 * h + 3] = w.w;
    }
}

// max of |v| on the bit patterns: a NaN counts above infinity instead of being dropped
__device__ __forceinline__ uint32_t abs_max(uint32_t m, const float (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    return m;
}

// A row's scale, amax after a multiplication by the power of two `pre`, and the factor
// pre * 127 / amax.
struct RowScale {
    float scale, pre, amax, factor;
};

// From the row's abs_max.  The power of two brings extreme rows to where 127 v and 1 / amax are
// normal numbers (what it pushes below the smallest one rounds to 0 anyway).  A row with a
// NaN or an infinity has scale NaN.
__device__ __forceinline__ RowScale row_scale(uint32_t m) {
    const float top = __uint_as_float(m);
    const bool finite = m < 0x7f800000u;
    RowScale s;
    s.pre = top > 0x1p100f ? 0x1p-64f : top < 0x1p-60f ? 0x1p64f : 1.f;
    s.amax = top * s.pre;
    s.factor = finite && top > 0.f ? 127.f * __frcp_rn(s.amax) : 0.f;
    s.scale = finite ? __fdiv_rn(top, 127.f) : __int_as_float(0x7fc00000);
    return s;
}

// rint(127 v / amax) of 16 values to q.  v * factor is within 2.3e-5 of the quotient (three
// roundings, 2^-24 each, of numbers up to 127); one that lands within 2.5e-5 of a tie is divided.
// (As a call for all 16, to keep the code short, the rare path cost decode batches 4 us: a
// warp takes it for 3% of its chunks.)  A row that is not finite is written as zeros.
__device__ __forceinline__ void store_chunk(int8_t* q, const float (&v)[16], const RowScale& s) {
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to the low bits
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (s.scale == s.scale) {
        uint32_t b[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float n = v[j] * s.pre, r = n * s.factor;
            float m = r + kRound;
            if (fabsf(r - (m - kRound)) > 0.5f - 2.5e-5f) m = __fdiv_rn(127.f * n, s.amax) + kRound;
            b[j] = __float_as_uint(m);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = __byte_perm(__byte_perm(b[4 * j], b[4 * j + 1], 0x0040),
                               __byte_perm(b[4 * j + 2], b[4 * j + 3], 0x0040), 0x5410);
    }
    *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace
}  // namespace moe
