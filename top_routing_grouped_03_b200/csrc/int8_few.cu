// int8_few.cu -- products of 8-bit integers for a handful of tokens (single-token serving): the
// formulas of int8_gemm.cu on the CUDA cores.
//
// Bound by the weights' bytes and by latency.  A tensor-core tile is 128 rows high and its
// pipeline (tensor maps, barriers, tensor memory, an epilogue per tile) costs 10 us before a
// 16 MB weight matrix has streamed past; here a warp owns whole weight rows, issues 16-byte
// loads for 4 KB of them at once, multiplies with dp4a against the tokens in shared memory and
// adds its lanes' int32 sums with one redux.sync.  The first loads are issued before the
// tokens are looked at, so that quantising them (every CTA for itself: a few KB) hides
// behind the weights' latency and costs no launch of its own.
//   * linear: 4096 x 4096, one token: 5.5 us (16.8 MB, 2.6 us of reading); the tensor cores took
//     12.9 and the rows' launch 2.3.
//   * experts: gate_up (h in fp32), the rows of h to 8 bits (quantize.cu), and down, which adds a
//     token's experts in registers in row order: no accumulator, no atomics, no combine: one
//     token, 8 experts of 1024 x 4096: 23.6 us with the token's own launch (101 MB, 15.5).  down
//     starts with gate_up and brings its weights into L2 until h is there.  (h quantised by
//     every CTA of down for itself, as linear does with its tokens, took 8 us longer than the
//     launch in between: 512 CTAs read the same 32 KB.)  Each (token, expert) row reads its
//     weights for itself, from L2 where rows share an expert; see few_experts_ok.
#include <algorithm>

#include "quantize.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
// CTAs to an SM, by registers: linear keeps 4 KB of weights a warp in them while it quantises the
// tokens (80 registers); the experts' kernels do not (64).
constexpr int kLinearCtas = 3, kExpertCtas = 4;
constexpr int kWarps = kThreads / 32;
constexpr int kChunkBytes = 512;  // of a weight row: 16 bytes a lane

__device__ __forceinline__ uint4 load_weights(const int8_t* p) {
    return __ldcs(reinterpret_cast<const uint4*>(p));  // read once
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int acc) {
    acc = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), acc);
    acc = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), acc);
    acc = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), acc);
    return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), acc);
}

__device__ __forceinline__ float scaled(int sum, float col_scale, float row_scale) {
    return row_scale * (__int2float_rn(sum) * col_scale);
}

// `rows` rows of `cols` values (a multiple of 16) as 8-bit integers to shared memory q (rows
// `stride` bytes apart) and their scales to `scale`; all threads of the CTA, per: warps to a row
// (a power of two).  part: one word per warp.
__device__ __forceinline__ void quantise_rows(const bf16* x, int rows, int cols, int8_t* q, int stride,
                                              float* scale, uint32_t* part, int per) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp & (per - 1), step = per * kChunkBytes;
    for (int r0 = 0; r0 < rows; r0 += kWarps / per) {
        const int r = r0 + warp / per;
        const int n = r < rows ? cols : 0;
        const bf16* row = x + static_cast<size_t>(r) * cols;
        const int c0 = (sub * 32 + lane) * 16;
        float first[16];
        uint32_t m = 0;
        if (c0 < n) {
            load_chunk(row + c0, first);
            m = abs_max(m, first);
        }
        for (int c = c0 + step; c < n; c += step) {
            float v[16];
            load_chunk(row + c, v);
            m = abs_max(m, v);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (per > 1) {
            __syncthreads();  // part is free
            if (lane == 0) part[warp] = m;
            __syncthreads();
            for (int w = 0; w < per; ++w) m = max(m, part[(warp & ~(per - 1)) + w]);
        }
        const RowScale s = row_scale(m);
        if (n > 0 && sub == 0 && lane == 0) scale[r] = s.scale();
        if (c0 < n) store_chunk(q + r * stride + c0, first, s);
        for (int c = c0 + step; c < n; c += step) {
            float v[16];
            load_chunk(row + c, v);
            store_chunk(q + r * stride + c, v, s);
        }
    }
}

// ---------------------------------------------------------------- linear

struct LinearArgs {
    const bf16* x;       // [T, K], or NULL: xq and x_scale are given
    const int8_t* xq;
    const float* x_scale;
    const int8_t* w;
    const float* w_scale;
    int T, N, K, stride; // stride: bytes of a token in shared memory
    bf16* out;
};

// R weight rows to a warp, C chunks of each in flight, up to TT tokens.
template <int R, int C, int TT>
__global__ void __launch_bounds__(kThreads, kLinearCtas) few_linear_kernel(LinearArgs a) {
    extern __shared__ __align__(16) int8_t sm[];
    __shared__ float s_scale[TT];
    __shared__ uint32_t s_part[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = (a.N + R - 1) / R;
    const int first = blockIdx.x * kWarps + warp, step = gridDim.x * kWarps;
    uint4 w[R][C];
    auto load = [&](int g, int k0) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int n = g * R + r, k = k0 + c * kChunkBytes + lane * 16;
                w[r][c] = n < a.N && k < a.K
                              ? load_weights(a.w + static_cast<size_t>(n) * a.K + k)
                              : make_uint4(0, 0, 0, 0);
            }
    };
    load(first, 0);  // (past the last group: zeros)
    if (a.x) {
        quantise_rows(a.x, a.T, a.K, sm, a.stride, s_scale, s_part, kWarps / TT);
    } else {
        for (int t = 0; t < a.T; ++t)
            for (int k = threadIdx.x * 16; k < a.K; k += kThreads * 16)
                *reinterpret_cast<uint4*>(sm + t * a.stride + k) =
                    __ldg(reinterpret_cast<const uint4*>(a.xq + static_cast<size_t>(t) * a.K + k));
        if (threadIdx.x < a.T) s_scale[threadIdx.x] = a.x_scale[threadIdx.x];
    }
    __syncthreads();
    for (int g = first; g < groups; g += step) {
        int acc[R][TT];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[r][t] = 0;
        for (int k0 = 0; k0 < a.K; k0 += C * kChunkBytes) {
            if (g != first || k0 != 0) load(g, k0);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + c * kChunkBytes + lane * 16;
                if (k >= a.K) break;  // (the weights there are zeros)
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    if (t >= a.T) break;
                    const uint4 x = *reinterpret_cast<const uint4*>(sm + t * a.stride + k);
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r][t] = dot16(w[r][c], x, acc[r][t]);
                }
            }
        }
        int mine = 0;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int s = __reduce_add_sync(0xffffffffu, acc[r][t]);
                if (lane == r * TT + t) mine = s;
            }
        const int n = g * R + lane / TT, t = lane % TT;
        if (lane < R * TT && n < a.N && t < a.T)
            a.out[static_cast<size_t>(t) * a.N + n] =
                __float2bfloat16_rn(scaled(mine, __ldg(a.w_scale + n), s_scale[t]));
    }
}

template <int TT>
cudaError_t launch_linear(const LinearArgs& a, int num_sms, cudaStream_t s) {
    const int chunks = ceil_div(a.K, kChunkBytes);
    const size_t smem = static_cast<size_t>(a.T) * a.stride;
    auto go = [&](auto kernel, int rows) {
        cudaError_t err = set_smem_limit(reinterpret_cast<const void*>(kernel), smem);
        if (err != cudaSuccess) return err;
        const int grid = std::min(ceil_div(ceil_div(a.N, rows), kWarps), kLinearCtas * num_sms);
        err = launch_kernel(kernel, dim3(grid), dim3(kThreads), smem, s, false, a);
        count_launches(1);
        return err;
    };
    if (chunks > 4) return go(few_linear_kernel<1, 8, TT>, 1);
    if (chunks > 2) return go(few_linear_kernel<2, 4, TT>, 2);
    if (chunks > 1 || TT == 8) return go(few_linear_kernel<4, 2, TT>, 4);
    return go(few_linear_kernel<8, 1, TT <= 4 ? TT : 4>, 8);
}

// ---------------------------------------------------------------- experts

// Expert and token of each row, from the offsets and sorted_token.
__device__ __forceinline__ int read_rows(const Int8FewExperts& a, int* s_expert, int* s_token) {
    const int rows = min(a.offsets[a.E], kFewRows);
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        const int hi = min(a.offsets[e + 1], rows);
        for (int r = max(a.offsets[e], 0); r < hi; ++r) s_expert[r] = e;
    }
    if (threadIdx.x < rows) s_token[threadIdx.x] = a.sorted_token[threadIdx.x];
    __syncthreads();
    return rows;
}

// h[row, j] = SiLU(g) u, a warp to a (row, feature): its gate and its up weight row.
__global__ void __launch_bounds__(kThreads, kExpertCtas) few_gate_up_kernel(Int8FewExperts a) {
    extern __shared__ __align__(16) int8_t sm[];  // the tokens [T, D]
    __shared__ int s_expert[kFewRows], s_token[kFewRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_launch();  // down may start on its weights
    if (a.status && blockIdx.x == 0 && threadIdx.x == 0) *a.status = MOE_OK;
    for (int i = threadIdx.x * 16; i < a.T * a.D; i += kThreads * 16)
        *reinterpret_cast<uint4*>(sm + i) = __ldg(reinterpret_cast<const uint4*>(a.xq + i));
    const int rows = read_rows(a, s_expert, s_token);
    constexpr int C = 4;
    const int total = rows * a.f;
    for (int u = blockIdx.x * kWarps + warp; u < total; u += gridDim.x * kWarps) {
        const int row = u / a.f, j = u - row * a.f;
        const int e = s_expert[row], t = s_token[row];
        const size_t gate_row = static_cast<size_t>(e) * 2 * a.f + j;
        const int8_t* wg = a.w_gate_up + gate_row * a.D;
        const int8_t* wu = wg + static_cast<size_t>(a.f) * a.D;
        const int8_t* x = sm + t * a.D;
        int g = 0, v = 0;
        for (int k0 = 0; k0 < a.D; k0 += C * kChunkBytes) {
            uint4 w[2][C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + c * kChunkBytes + lane * 16;
                w[0][c] = k < a.D ? load_weights(wg + k) : make_uint4(0, 0, 0, 0);
                w[1][c] = k < a.D ? load_weights(wu + k) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + c * kChunkBytes + lane * 16;
                if (k >= a.D) break;
                const uint4 xv = *reinterpret_cast<const uint4*>(x + k);
                g = dot16(w[0][c], xv, g);
                v = dot16(w[1][c], xv, v);
            }
        }
        g = __reduce_add_sync(0xffffffffu, g);
        v = __reduce_add_sync(0xffffffffu, v);
        if (lane == 0) {
            const float rs = __ldg(a.x_scale + t);
            const float gs = scaled(g, __ldg(a.gate_up_scale + gate_row), rs);
            const float us = scaled(v, __ldg(a.gate_up_scale + gate_row + a.f), rs);
            a.h[static_cast<size_t>(row) * a.f + j] = __fdividef(gs, 1.f + __expf(-gs)) * us;
        }
    }
}

// out[t, d] = bf16(residual + sum over t's rows of weight * (W_down h)[d]), a warp to an output
// feature d: R rows' weight rows in flight, C chunks of each; lane r then holds row r's sum, and
// lane t adds up token t's rows in order.
template <int R, int C>
__global__ void __launch_bounds__(kThreads, kExpertCtas) few_down_kernel(Int8FewExperts a) {
    extern __shared__ __align__(16) int8_t sm[];  // h as 8-bit integers [rows, f]
    __shared__ int s_expert[kFewRows], s_token[kFewRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = read_rows(a, s_expert, s_token);  // (older than gate_up's launch)
    const int my_row = min(lane, kFewRows - 1);
    const size_t my_scale = lane < rows ? static_cast<size_t>(s_expert[my_row]) * a.D : 0;
    const int first = blockIdx.x * kWarps + warp, step = gridDim.x * kWarps;
    // this warp's weights towards L2 while gate_up finishes: 128-byte lines
    for (int d = first; d < a.D; d += step)
        for (int r = 0; r < rows; ++r)
            for (int k = lane * 128; k < a.f; k += 32 * 128)
                prefetch_l2(a.w_down + (static_cast<size_t>(s_expert[r]) * a.D + d) * a.f + k);
    uint4 w[R][C];
    auto load = [&](int d, int r0, int k0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int8_t* row = r0 + r < rows
                                    ? a.w_down + (static_cast<size_t>(s_expert[r0 + r]) * a.D + d) * a.f
                                    : nullptr;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int k = k0 + c * kChunkBytes + lane * 16;
                w[r][c] = row && k < a.f ? load_weights(row + k) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    grid_dep_wait();  // the rows of h
    for (int i = threadIdx.x * 16; i < rows * a.f; i += kThreads * 16)
        *reinterpret_cast<uint4*>(sm + i) = __ldcg(reinterpret_cast<const uint4*>(a.hq + i));
    const float row_factor = lane < rows ? __ldcg(a.hs + my_row) * a.sorted_w[my_row] : 0.f;
    __syncthreads();
    for (int d = first; d < a.D; d += step) {
        const float cs = lane < rows ? __ldg(a.down_scale + my_scale + d) : 0.f;
        float y = 0.f;
        if (lane < a.T && a.residual)
            y = __bfloat162float(a.residual[static_cast<size_t>(lane) * a.D + d]);
        int mine = 0;
        for (int r0 = 0; r0 < rows; r0 += R) {
            int acc[R];
#pragma unroll
            for (int r = 0; r < R; ++r) acc[r] = 0;
            for (int k0 = 0; k0 < a.f; k0 += C * kChunkBytes) {
                load(d, r0, k0);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r0 + r >= rows) break;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const int k = k0 + c * kChunkBytes + lane * 16;
                        if (k >= a.f) break;
                        acc[r] = dot16(w[r][c], *reinterpret_cast<const uint4*>(sm + (r0 + r) * a.f + k),
                                       acc[r]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int sum = __reduce_add_sync(0xffffffffu, acc[r]);
                if (lane == r0 + r) mine = sum;
            }
        }
        const float v = scaled(mine, cs, row_factor);
        for (int r = 0; r < rows; ++r) {
            const float vr = __shfl_sync(0xffffffffu, v, r);
            if (lane == s_token[r]) y += vr;
        }
        if (lane < a.T) a.out[static_cast<size_t>(lane) * a.D + d] = __float2bfloat16_rn(y);
    }
}

}  // namespace

// Up to 8 tokens, as far as they fit in shared memory.  us here against the tiles with their rows'
// launch, by tokens (weights from HBM): 1024 x 1024 1: 2.7/8.0, 8: 4.8/7.9; 4096 x 4096 1: 6.3/20.1,
// 4: 10.1/19.7, 8: 15.9/18.6.  A token costs a dp4a for every four weights, so larger matrices cross
// earlier: 4096 x 8192 4: 17.4/20.8, 5: 22.9/21.0, 8: 29.1/20.5; 14336 x 4096 4: 17.5/22.6, 5:
// 22.5/22.1, 8: 31.3/21.4.  The limit does not follow them: callers rely on it for calls without a
// workspace.
bool few_linear_ok(int T, int K) {
    return T <= 8 && static_cast<long long>(T) * ((K + 15) & ~15) <= 65536;
}

cudaError_t launch_few_linear(const bf16* x, const int8_t* xq, const float* x_scale, const int8_t* w,
                              const float* w_scale, int T, int N, int K, bf16* out, int num_sms,
                              cudaStream_t s) {
    const LinearArgs a{x, xq, x_scale, w, w_scale, T, N, K, K, out};
    return T == 1   ? launch_linear<1>(a, num_sms, s)
           : T == 2 ? launch_linear<2>(a, num_sms, s)
           : T <= 4 ? launch_linear<4>(a, num_sms, s)
                    : launch_linear<8>(a, num_sms, s);
}

// Up to 16 rows.  us here against weights on M, 128 experts of D 2048, f 512 and of 4096, 1024: 8 rows of
// one token 12.4/24.2 and 23.9/35.4; 16 rows of 2 tokens 18.1/26.6 and 41.2/48.8; 16 tokens with an
// expert each 19.0/26.6 and 49.9/48.9, all with the same expert 17.3/24.6 and 33.5/32.8.
bool few_experts_ok(int T, int D, int K, int f) {
    const long long rows = static_cast<long long>(T) * K;
    return rows <= kFewRows && static_cast<long long>(T) * D <= 65536 && rows * f <= 65536;
}

cudaError_t launch_few_experts(const Int8FewExperts& a, int num_sms, cudaStream_t s) {
    const int rows = a.T * a.K, chunks = ceil_div(a.f, kChunkBytes);
    auto go = [&](auto kernel, int warps, size_t smem, bool pdl) {
        cudaError_t err = set_smem_limit(reinterpret_cast<const void*>(kernel), smem);
        if (err != cudaSuccess) return err;
        err = launch_kernel(kernel, dim3(std::min(ceil_div(warps, kWarps), kExpertCtas * num_sms)),
                            dim3(kThreads), smem, s, pdl, a);
        count_launches(1);
        return err;
    };
    cudaError_t err = go(few_gate_up_kernel, rows * a.f, static_cast<size_t>(a.T) * a.D, false);
    if (err != cudaSuccess) return err;
    QuantizeLaunch q{};
    q.x = a.h;
    q.is_f32 = true;
    q.rows = rows;
    q.cols = a.f;
    q.q = a.hq;
    q.scale = a.hs;
    q.row_count = a.offsets + a.E;
    if ((err = launch_quantize(q, s, true)) != cudaSuccess) return err;
    const size_t smem = static_cast<size_t>(rows) * a.f;
    return chunks == 1   ? go(few_down_kernel<8, 1>, a.D, smem, true)
           : chunks == 2 ? go(few_down_kernel<4, 2>, a.D, smem, true)
                         : go(few_down_kernel<2, 4>, a.D, smem, true);
}

}  // namespace moe
