// quantize.cu -- rows of activations (or weights) to 8-bit integers with one scale per row.
//
//   amax_r = max_c |x[r, c]|,  q[r, c] = rint(127 x[r, c] / amax_r),  scale[r] = amax_r / 127
// (rint: to nearest, ties to even), so that x ~ q scale and |q| <= 127.  The quotient of
// 127 x and amax, correctly rounded to fp32, decides: for bf16 x both are exact and the
// quotient is never rounded onto a tie, so q is the exact rounding of the real quotient.
// Most elements take a product with 1 / amax instead, which is within 3e-5 of the quotient;
// only one that lands within 6e-5 of a tie is divided.
//
// Bound by memory: a row is read once (kept in registers between the maximum and the
// rounding up to kKeep chunks a thread) and written once.  A warp takes a row of up to 2048
// columns, a CTA a longer one.
#include <cmath>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16;  // columns of one thread at a time: one 16-byte store
constexpr int kKeep = 4;    // chunks a thread keeps in registers

// 16 values as fp32
__device__ __forceinline__ void load_chunk(const bf16* p, float (&v)[kChunk]) {
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
__device__ __forceinline__ void load_chunk(const float* p, float (&v)[kChunk]) {
    const float4* s = reinterpret_cast<const float4*>(p);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float4 w = __ldcg(s + h);
        v[4 * h] = w.x; v[4 * h + 1] = w.y; v[4 * h + 2] = w.z; v[4 * h + 3] = w.w;
    }
}

// max of |v| on the bit patterns: a NaN counts above infinity instead of being dropped
__device__ __forceinline__ uint32_t abs_max(uint32_t m, const float (&v)[kChunk]) {
#pragma unroll
    for (int j = 0; j < kChunk; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    return m;
}

struct RowScale {
    float amax, inv, pre;
};

// rint(127 v / amax) in the low byte of the result (two's complement)
__device__ __forceinline__ uint32_t quantise(float v, const RowScale& s) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number
    const float n = 127.f * (v * s.pre);
    const float r = n * s.inv;
    float m = r + kMagic;
    if (fabsf(fabsf(r - (m - kMagic)) - 0.5f) < 6e-5f) m = __fdiv_rn(n, s.amax) + kMagic;
    return __float_as_uint(m) & 0xffu;
}

__device__ __forceinline__ void store_chunk(int8_t* q, const float (&v)[kChunk], const RowScale& s) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = quantise(v[4 * j], s) | (quantise(v[4 * j + 1], s) << 8) |
               (quantise(v[4 * j + 2], s) << 16) | (quantise(v[4 * j + 3], s) << 24);
    *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
}

// kRowThreads threads (a warp or the CTA) take one row.
template <typename T, int kRowThreads>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(QuantizeLaunch a) {
    __shared__ uint32_t s_max[kThreads / 32];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x % kRowThreads;
    if (a.clear && blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.clear_words; i += kThreads) a.clear[i] = 0u;
    const long long row =
        static_cast<long long>(blockIdx.x) * (kThreads / kRowThreads) + threadIdx.x / kRowThreads;
    const long long rows = a.row_count ? min(static_cast<long long>(*a.row_count), a.rows) : a.rows;
    if (row >= rows) return;  // whole warps, or the whole CTA
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.cols;
    int8_t* q = a.q + row * a.cols;
    constexpr int kStep = kRowThreads * kChunk;
    float keep[kKeep][kChunk];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int c = lane * kChunk + k * kStep;
        if (c < a.cols) {
            load_chunk(x + c, keep[k]);
            m = abs_max(m, keep[k]);
        }
    }
    for (int c = lane * kChunk + kKeep * kStep; c < a.cols; c += kStep) {
        float v[kChunk];
        load_chunk(x + c, v);
        m = abs_max(m, v);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (kRowThreads > 32) {
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
        __syncthreads();
        m = s_max[0];
#pragma unroll
        for (int w = 1; w < kThreads / 32; ++w) m = max(m, s_max[w]);
    }
    // A power of two brings extreme rows to where 127 v and 1 / amax are normal numbers (what it
    // pushes below the smallest one rounds to 0 anyway).  inv = 0 rounds the row to zeros: for a
    // zero row, and for one with a NaN or an infinity (0 * those is NaN: the low byte of NaN's
    // bit pattern is 0xff, so such rows are written as zeros explicitly).
    const float top = __uint_as_float(m);
    const bool finite = m < 0x7f800000u;
    RowScale s;
    s.pre = top > 0x1p100f ? 0x1p-64f : top < 0x1p-60f ? 0x1p64f : 1.f;
    s.amax = top * s.pre;
    s.inv = finite && top > 0.f ? __frcp_rn(s.amax) : 0.f;
    if (lane == 0) a.scale[row] = finite ? __fdiv_rn(top, 127.f) : __int_as_float(0x7fc00000);
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        const int c = lane * kChunk + k * kStep;
        if (c >= a.cols) break;
        if (finite) store_chunk(q + c, keep[k], s);
        else *reinterpret_cast<uint4*>(q + c) = make_uint4(0, 0, 0, 0);
    }
    for (int c = lane * kChunk + kKeep * kStep; c < a.cols; c += kStep) {
        float v[kChunk];
        load_chunk(x + c, v);
        if (finite) store_chunk(q + c, v, s);
        else *reinterpret_cast<uint4*>(q + c) = make_uint4(0, 0, 0, 0);
    }
}

template <typename T>
cudaError_t launch_typed(const QuantizeLaunch& a, cudaStream_t s, bool pdl) {
    const bool by_warp = a.cols <= 32 * kChunk * kKeep;
    const long long per = by_warp ? kThreads / 32 : 1;
    const dim3 grid(static_cast<unsigned>((a.rows + per - 1) / per));
    return by_warp ? launch_kernel(quantize_rows_kernel<T, 32>, grid, dim3(kThreads), 0, s, pdl, a)
                   : launch_kernel(quantize_rows_kernel<T, kThreads>, grid, dim3(kThreads), 0, s,
                                   pdl, a);
}

}  // namespace

cudaError_t launch_quantize(const QuantizeLaunch& a, cudaStream_t s, bool pdl) {
    if (a.rows == 0) return cudaSuccess;
    const cudaError_t err = a.is_f32 ? launch_typed<float>(a, s, pdl) : launch_typed<bf16>(a, s, pdl);
    count_launches(1);
    return err;
}

}  // namespace moe
