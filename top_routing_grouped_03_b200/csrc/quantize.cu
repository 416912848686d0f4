// quantize.cu -- rows of activations (or weights) to 8-bit integers with one scale per row.
//
//   amax_r = max_c |x[r, c]|,  q[r, c] = rint(127 x[r, c] / amax_r),  scale[r] = amax_r / 127
// (rint: to nearest, ties to even), so that x ~ q scale and |q| <= 127.  The quotient of
// 127 x and amax, correctly rounded to fp32, decides: for bf16 x both are exact and the
// quotient is never rounded onto a tie, so q is the exact rounding of the real quotient.
// Most elements take a product with 127 / amax instead, which is within 4.6e-5 of the
// quotient; those within 5e-5 of a tie are divided.
//
// Bound by memory: a row is read once (kept in registers between the maximum and the
// rounding) and written once.  As many threads take a row as give each 16 columns, from a warp
// to a CTA: with a warp to every row of up to 2048 columns and four chunks kept, the registers
// left a third of the warps (8192 x 4096 bf16: 57 us).  Now 26 us (101 MB, 15 us of copying: CTAs of
// one row come and go too fast to keep the loads queued), 65536 x 1024 fp32 rows 56 us (336 MB, 52).
#include "quantize.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 16;  // columns of one thread at a time

// A thread's 16 columns are pieces of one 16-byte load, a piece of every thread of the row after
// another, so that a warp's loads (through L2 only) and stores cover whole sectors: with 16
// columns in a row per thread fp32 rows were fetched twice from L2 (65536 x 1024: 73 against 70 us).
template <typename T>
constexpr int kPiece = 16 / sizeof(T);

__device__ __forceinline__ void load_piece(const bf16* p, float* v) {
    const uint4 w = __ldcg(reinterpret_cast<const uint4*>(p));
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}
__device__ __forceinline__ void load_piece(const float* p, float* v) {
    const float4 w = __ldcg(reinterpret_cast<const float4*>(p));
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
}

// Columns c0 + [0, kChunk * threads) of a row of cols, this thread's share (zeros past the row).
template <int kRowThreads, typename T>
__device__ __forceinline__ void load_share(const T* x, int c0, int cols, int lane, float (&v)[kChunk]) {
#pragma unroll
    for (int k = 0; k < kChunk; k += kPiece<T>) {
        const int c = c0 + k * kRowThreads + lane * kPiece<T>;
        if (c < cols) {
            load_piece(x + c, v + k);
        } else {
#pragma unroll
            for (int j = 0; j < kPiece<T>; ++j) v[k + j] = 0.f;
        }
    }
}
template <int kRowThreads, typename T>
__device__ __forceinline__ void store_share(int8_t* q, int c0, int cols, int lane,
                                            const float (&v)[kChunk], const RowScale& s) {
#pragma unroll
    for (int k = 0; k < kChunk; k += kPiece<T>) {
        const int c = c0 + k * kRowThreads + lane * kPiece<T>;
        if (c >= cols) continue;
        if (kPiece<T> == 8)
            *reinterpret_cast<uint2*>(q + c) = make_uint2(quantise4(v + k, s), quantise4(v + k + 4, s));
        else
            *reinterpret_cast<uint32_t*>(q + c) = quantise4(v + k, s);
    }
}

// kRowThreads threads take one row; a thread keeps kKeep chunks, longer rows are read again
// past them.
template <typename T, int kRowThreads, int kKeep>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(QuantizeLaunch a) {
    __shared__ uint32_t s_max[kThreads / 32];
    grid_dep_launch();  // what follows may start up to its own wait
    grid_dep_wait();
    const int lane = threadIdx.x % kRowThreads;
    if (a.clear && blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.clear_words; i += kThreads) a.clear[i] = 0u;
    const long long row =
        static_cast<long long>(blockIdx.x) * (kThreads / kRowThreads) + threadIdx.x / kRowThreads;
    const long long rows = a.row_count ? min(static_cast<long long>(*a.row_count), a.rows) : a.rows;
    const int cols = row < rows ? a.cols : 0;  // a thread without a row goes along to the barrier
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.cols;
    int8_t* q = a.q + row * a.cols;
    constexpr int kStep = kRowThreads * kChunk;
    float keep[kKeep][kChunk];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
        load_share<kRowThreads>(x, k * kStep, cols, lane, keep[k]);
        m = abs_max(m, keep[k]);
    }
    for (int c = kKeep * kStep; c < cols; c += kStep) {
        float v[kChunk];
        load_share<kRowThreads>(x, c, cols, lane, v);
        m = abs_max(m, v);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (kRowThreads > 32) {
        const int warp = threadIdx.x >> 5, first = warp & ~(kRowThreads / 32 - 1);
        if ((threadIdx.x & 31) == 0) s_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kRowThreads / 32; ++w) m = max(m, s_max[first + w]);
    }
    if (cols == 0) return;
    const RowScale s = row_scale(m);
    if (lane == 0) a.scale[row] = s.scale();
#pragma unroll
    for (int k = 0; k < kKeep; ++k) store_share<kRowThreads, T>(q, k * kStep, cols, lane, keep[k], s);
    for (int c = kKeep * kStep; c < cols; c += kStep) {
        float v[kChunk];
        load_share<kRowThreads>(x, c, cols, lane, v);
        store_share<kRowThreads, T>(q, c, cols, lane, v, s);
    }
}

template <typename T>
cudaError_t launch_typed(const QuantizeLaunch& a, cudaStream_t s, bool pdl) {
    int threads = 32;
    while (threads < kThreads && threads * kChunk < a.cols) threads *= 2;
    const long long per = kThreads / threads;
    const dim3 grid(static_cast<unsigned>((a.rows + per - 1) / per));
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kThreads), 0, s, pdl, a); };
    return threads == 32    ? go(quantize_rows_kernel<T, 32, 1>)
           : threads == 64  ? go(quantize_rows_kernel<T, 64, 1>)
           : threads == 128 ? go(quantize_rows_kernel<T, 128, 1>)
           : a.cols <= kThreads * kChunk ? go(quantize_rows_kernel<T, kThreads, 1>)
                                         : go(quantize_rows_kernel<T, kThreads, 2>);
}

}  // namespace

cudaError_t launch_quantize(const QuantizeLaunch& a, cudaStream_t s, bool pdl) {
    if (a.rows == 0) return cudaSuccess;
    const cudaError_t err = a.is_f32 ? launch_typed<float>(a, s, pdl) : launch_typed<bf16>(a, s, pdl);
    count_launches(1);
    return err;
}

}  // namespace moe
