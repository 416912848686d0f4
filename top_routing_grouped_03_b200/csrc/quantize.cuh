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

// rint(127 v / amax) in the low byte of the result (two's complement).  v * factor is within 2.3e-5
// of the quotient (three roundings, 2^-24 each, of numbers up to 127); one that lands within
// 2.5e-5 of a tie is divided.  (A call for 16 values at a time, to keep the code short, cost decode
// batches 4 us: a warp takes the rare path for 3% of its 512 values.)
__device__ __forceinline__ uint32_t quantise(float v, const RowScale& s) {
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to the low bits
    const float n = v * s.pre, r = n * s.factor;
    float m = r + kRound;
    if (fabsf(r - (m - kRound)) > 0.5f - 2.5e-5f) m = __fdiv_rn(127.f * n, s.amax) + kRound;
    return __float_as_uint(m);
}

// Four values as bytes; zeros in a row that is not finite.
__device__ __forceinline__ uint32_t quantise4(const float* v, const RowScale& s) {
    if (s.scale != s.scale) return 0u;
    return __byte_perm(__byte_perm(quantise(v[0], s), quantise(v[1], s), 0x0040),
                       __byte_perm(quantise(v[2], s), quantise(v[3], s), 0x0040), 0x5410);
}

__device__ __forceinline__ void store_chunk(int8_t* q, const float (&v)[16], const RowScale& s) {
    *reinterpret_cast<uint4*>(q) =
        make_uint4(quantise4(v, s), quantise4(v + 4, s), quantise4(v + 8, s), quantise4(v + 12, s));
}

}  // namespace
}  // namespace moe
