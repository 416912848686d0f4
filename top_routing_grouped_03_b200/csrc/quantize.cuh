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

// The bits of max |v| (m: those of a maximum so far), which order like the numbers; a NaN counts
// above infinity instead of being dropped.
__device__ __forceinline__ uint32_t abs_max(uint32_t m, const float (&v)[16]) {
    float f = __uint_as_float(m);
#pragma unroll
    for (int j = 0; j < 16; j += 2) f = max_nan3(f, v[j], v[j + 1]);
    return __float_as_uint(f);
}

// What rounds a row's values: `top` its abs_max, amax = top * pre with a power of two, and
// pre * 127 / top.  The power of two brings extreme rows to where 127 v and 1 / amax are normal
// numbers (what it pushes below the smallest one rounds to 0 anyway).
struct RowScale {
    float top, pre, amax, factor;
    bool finite;

    // the row's scale: NaN in a row with a NaN or an infinity.  (A division: for one thread of a
    // row; by all of them it was a fifth of the kernel's instructions.)
    __device__ __forceinline__ float scale() const {
        return finite ? __fdiv_rn(top, 127.f) : __int_as_float(0x7fc00000);
    }
};

__device__ __forceinline__ RowScale row_scale(uint32_t m) {
    RowScale s;
    s.top = __uint_as_float(m);
    s.finite = m < 0x7f800000u;
    s.pre = s.top > 0x1p100f ? 0x1p-64f : s.top < 0x1p-60f ? 0x1p64f : 1.f;
    s.amax = s.top * s.pre;
    float inv;  // within 2^-22 of 1 / amax (documented: 2^-23 where 1 / amax is 1/2 to 1)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s.amax));
    s.factor = s.finite && s.top > 0.f ? 127.f * inv : 0.f;
    return s;
}

// rint(127 v / amax) of four values, as bytes; zeros in a row that is not finite.  v * factor is
// within 4.6e-5 of the quotient (numbers up to 127 with 2^-22 from the reciprocal and 2^-24 from
// each product); where one of the four lands within 5e-5 of a tie they are divided.  One test for four values instead of one
// each, and one maximum for two: 20 -> 16 instructions a value, which bound the bf16 rows.
// (A call for 16 values, to keep the code short, cost decode batches 4 us: a warp takes
// the rare path for 5% of its chunks of 512 values.)
__device__ __forceinline__ uint32_t quantise4(const float* v, const RowScale& s) {
    constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to the low bits
    float n[4], m[4], off = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        n[j] = v[j] * s.pre;
        const float r = n[j] * s.factor;
        m[j] = r + kRound;
        off = fmaxf(off, fabsf(r - (m[j] - kRound)));
    }
    if (off > 0.5f - 5e-5f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = __fdiv_rn(127.f * n[j], s.amax) + kRound;
    }
    const uint32_t q = __byte_perm(__byte_perm(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0040),
                                   __byte_perm(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0040), 0x5410);
    return s.finite ? q : 0u;
}

__device__ __forceinline__ void store_chunk(int8_t* q, const float (&v)[16], const RowScale& s) {
    *reinterpret_cast<uint4*>(q) =
        make_uint4(quantise4(v, s), quantise4(v + 4, s), quantise4(v + 8, s), quantise4(v + 12, s));
}

}  // namespace
}  // namespace moe
