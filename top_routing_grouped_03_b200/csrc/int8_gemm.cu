// int8_gemm.cu -- products of 8-bit integers with a scale for each token and each weight row:
//   y[t, n] = xs[t] ws[n] sum_k xq[t, k] wq[n, k]
// grouped over experts (gate_up with SwiGLU, down with the routing weights) or dense, on the
// kernels of grouped_gemm.cuh with tcgen05.mma.kind::i8: the sums are int32 and exact, the
// scales are applied once per element in the epilogue.
//
// Against bf16 a weight takes half the bytes (what bounds few tokens: HBM) and the tensor
// cores do twice the products (what bounds many tokens).  Weights on M for groups of a handful
// of rows, one-CTA tiles of 128 tokens x 256 weight rows above (K cut into slices when the
// tiles cannot fill the GPU), CTA pairs (256 x 256) once groups average 128 rows.
//
// gate_up leaves h in fp32: its row maxima are known only when all feature blocks are done.
// (Letting the CTA that completes a row block quantise it, from L2, saved a launch but was bound
// by the latency of one CTA's loads: 65536 x 1024 rows 436 -> 1640 us.)
//
// Measured: dense 8192 x 8192 x 4096 171 us (3.2 Pop/s); prompt experts (65536 rows, 64 experts,
// 4096 x 1024) gate_up 414 us (2.66 Pop/s, 81% of the tensor pipe), down 292 us (bound by its
// 570 MB of rows out of the epilogue); fine-grained gate_up (80 rows a group, 512 groups) 691 us,
// 6.2 TB/s of weights.  Gathering the token rows with TMA (tile::gather4) instead of a copy
// before CTA pairs or cp.async in one-CTA tiles: the prompt experts 1010 to 2230 us, 1021
// skewed tokens 84 to 148 us.
#include <algorithm>

#include "grouped_gemm.cuh"

namespace moe {
namespace {

// Rows in expert order for the CTA-pair kernel: out[r] = x[tok[r]] for r < *row_count, a warp to
// a row, four 16-byte loads of each lane in flight.
__global__ void __launch_bounds__(256) gather_rows_i8_kernel(const uint4* x, const int32_t* tok,
                                                             const int32_t* row_count, int rows,
                                                             int vec, uint4* out) {
    grid_dep_wait();
    grid_dep_launch();
    const int n = row_count ? min(*row_count, rows) : rows;
    const int lane = threadIdx.x & 31;
    for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r < n; r += gridDim.x * 8) {
        const uint4* src = x + static_cast<size_t>(__ldg(tok + r)) * vec;
        uint4* dst = out + static_cast<size_t>(r) * vec;
        for (int i0 = lane; i0 < vec; i0 += 128) {
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + 32 * u < vec) v[u] = __ldg(src + i0 + 32 * u);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + 32 * u < vec) dst[i0 + 32 * u] = v[u];
        }
    }
}

// CTA pairs for groups of 128 rows and more, if one group's pair tiles fill at least half of
// the pairs (333 x 2048 x 4096 has 16 of them: 20 us in pairs).
bool use_pairs(const Int8GemmLaunch& a, int num_sms) {
    if (a.E == 1) {
        const int cols = a.kind == Int8GemmLaunch::kGateUp ? 2 * a.f : a.D;
        if (4ll * ceil_div(a.rows, CfgPair::kPairRows) * ceil_div(cols, kTmN) < num_sms) return false;
    }
    const bool gathered = a.kind == Int8GemmLaunch::kGateUp && a.sorted_token != nullptr;
    return num_sms >= 2 && a.rows / a.E >= 128 && (!gathered || a.gather_buf != nullptr);
}

// Weight rows of a one-CTA tile.  Tiles of 256 rows reuse a token row most; when one group's
// tiles cannot fill half of the GPU, narrower ones spread the weights over more SMs, which
// costs less than cutting K into slices whose sums meet in memory (77 x 4104 x 2064 with its
// rows' quantisation: 30 us with 256 rows and 4 slices, 11.6 with 64 rows).
int tile_width(const Int8GemmLaunch& a, int num_sms) {
    if (a.E != 1 || a.kind == Int8GemmLaunch::kDown) return kTmN;
    const long long blocks = ceil_div(a.rows, kTmRows);
    const int cols = a.kind == Int8GemmLaunch::kGateUp ? 2 * a.f : a.D;
    for (int wn = kTmN; wn > 64; wn /= 2)
        if (2 * blocks * ceil_div(cols, wn) > num_sms) return wn;
    return 64;
}

// Weights on M (128 weight rows x 32 token rows) while the groups average a handful of rows: all
// epilogue warps then have features to drain, where a 128-row tile of tokens leaves the two
// or three rows of a group to one quarter of them (64 tokens, 256 experts, 8 each: 134.8 with tokens
// on M, 130.8 us; 8 tokens, 128 experts of 1024 x 4096: 165 to 134 us; 16-row tiles the same).
// Above, and with skewed routing, tokens on M read hot experts' weights fewer times (300 tokens,
// 9 rows a group on average, Zipf: 43 against 56 us).
constexpr int kSwapRows = 32;
bool use_swap(const Int8GemmLaunch& a) {
    return a.kind != Int8GemmLaunch::kDense && a.E > 1 && a.rows / a.E <= 8;
}

template <bool GATE_UP>
cudaError_t launch_swap(const CUtensorMap& mw, const CUtensorMap& ma, const Params& p, int ctas,
                        cudaStream_t s, bool pdl) {
    using C = Cfg<kSwapRows, GATE_UP>;
    const size_t smem = 1024 + static_cast<size_t>(C::kStages) * C::kStageBytes + (2 * C::kStages + 5) * 8 +
                        16 + 2 * (p.G + 1) * sizeof(int);
    auto kfn = grouped_gemm_kernel<kSwapRows, GATE_UP, true>;
    cudaError_t err = set_smem_limit(reinterpret_cast<const void*>(kfn), smem);
    if (err != cudaSuccess) return err;
    err = launch_kernel(kfn, dim3(ctas), dim3(kThreads), smem, s, pdl, mw, ma, p);
    count_launches(1);
    return err;
}

template <bool GATE_UP>
cudaError_t launch_one(const CUtensorMap& mw, const CUtensorMap& ma, const Params& p, bool pair, int wn,
                       int ctas, cudaStream_t s, bool pdl) {
    using P = CfgPair;
    const int stages = pair        ? P::kStages
                       : wn == 256 ? CfgTm<256>::kStages
                       : wn == 128 ? CfgTm<128>::kStages
                                   : CfgTm<64>::kStages;
    const int stage_bytes = pair        ? P::kStageBytes
                            : wn == 256 ? CfgTm<256>::kStageBytes
                            : wn == 128 ? CfgTm<128>::kStageBytes
                                        : CfgTm<64>::kStageBytes;
    const size_t smem = 1024 + static_cast<size_t>(stages) * stage_bytes + (2 * stages + 5) * 8 + 16 +
                        2 * (p.G + 1) * sizeof(int) + kI8EpilogueBytes;
    auto kfn = pair        ? grouped_gemm_pair_kernel<GATE_UP, true>
               : wn == 256 ? grouped_gemm_tm_kernel<GATE_UP, true, 256>
               : wn == 128 ? grouped_gemm_tm_kernel<GATE_UP, true, 128>
                           : grouped_gemm_tm_kernel<GATE_UP, true, 64>;
    cudaError_t err = set_smem_limit(reinterpret_cast<const void*>(kfn), smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kTmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pair) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = 2;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    err = cudaLaunchKernelEx(&cfg, kfn, mw, ma, p);
    count_launches(1);
    return err;
}

}  // namespace


bool int8_gemm_uses_pairs(const Int8GemmLaunch& a, int num_sms) { return use_pairs(a, num_sms); }

cudaError_t launch_int8_gemm(const Int8GemmLaunch& a, int num_sms, cudaStream_t s, bool pdl) {
    if (a.rows == 0) return cudaSuccess;
    if (a.E > kMaxGroups) return cudaErrorInvalidValue;
    const bool gate_up = a.kind == Int8GemmLaunch::kGateUp;
    const bool dense = a.kind == Int8GemmLaunch::kDense;
    const bool pair = use_pairs(a, num_sms);
    const int K = gate_up ? a.D : a.f;  // 8-bit values; the tensor maps count pairs of them
    const int w_group_rows = gate_up ? 2 * a.f : a.D;
    bool gather = gate_up && a.sorted_token != nullptr;
    const int8_t* act = a.act;
    cudaError_t err;
    if (pair && gather) {
        const int vec = K / 16;
        err = launch_kernel(gather_rows_i8_kernel, dim3(std::min(ceil_div(a.rows, 8), 8 * num_sms)),
                            dim3(256), 0, s, pdl, reinterpret_cast<const uint4*>(act), a.sorted_token,
                            a.offsets ? a.offsets + a.E : nullptr, a.rows, vec,
                            reinterpret_cast<uint4*>(a.gather_buf));
        count_launches(1);
        if (err != cudaSuccess) return err;
        act = a.gather_buf;
        gather = false;
        pdl = true;
    }
    CUtensorMap mw, ma;
    const bool swap = !pair && use_swap(a);
    const int wn = pair || swap ? kTmN : tile_width(a, num_sms);
    if ((err = encode_tile_map(&mw, a.w, static_cast<uint64_t>(w_group_rows) * a.E, K / 2, swap ? kBM : wn / 2)) !=
        cudaSuccess)
        return err;
    // with a gather the activation map is not read: it covers the first row
    if ((err = encode_tile_map(&ma, act, gather ? 1 : a.rows, K / 2, gather ? 1 : swap ? kSwapRows : kTmRows)) != cudaSuccess)
        return err;
    Params p{};
    p.offsets = a.offsets;
    p.rows_total = a.rows;
    p.sorted_token = a.sorted_token;
    p.sorted_w = a.sorted_w;
    p.G = a.E;
    p.nf = swap ? (gate_up ? a.f : a.D) / kBM : gate_up ? a.f / (wn / 2) : ceil_div(a.D, wn);
    p.nk = ceil_div(K, 2 * kBK);
    p.w_group_rows = w_group_rows;
    p.up_rows = a.f;
    p.out_cols = gate_up ? a.f : a.D;
    p.acc_out = a.acc_out;
    p.y_out = a.y_out;
    p.y16_out = a.y16_out;
    p.y16q_out = pair ? a.y16q_out : nullptr;
    p.y16q_scale = a.y16q_scale;
    p.status = a.status;
    p.gather_tok = gather ? a.sorted_token : nullptr;
    p.x = reinterpret_cast<const bf16*>(act);
    p.ksplit = 1;
    p.act_box = kSwapRows;
    p.zero_acc = gate_up ? a.zero_acc : nullptr;
    p.zero_n4 = a.zero_floats / 4;
    p.row_scale = a.act_scale;
    p.scale_tok = gate_up ? a.sorted_token : nullptr;
    p.col_scale = a.w_scale;
    p.h32_out = a.h_out;
    p.dense = dense ? 1 : 0;
    // gate_up and dense slices meet in the partial-sum planes; down's add into acc_out
    const bool split = !pair && !swap && a.ksplit_max > 1 &&
                       (a.kind == Int8GemmLaunch::kDown
                            ? (a.acc_out != nullptr && a.y_out == nullptr && a.y16_out == nullptr)
                            : (a.part != nullptr && a.tickets != nullptr && a.ticket_cap > 0));
    // A dense product's slices cost a round trip of partial sums; they pay where few tiles have a
    // long K (100 x 512 x 8192: 21 against 26 us; 77 x 4104 x 2064 the other way: 15 against 11),
    // and for up to half as many tiles as SMs where it is twice as long (16 x 4096 x 8192: 18.5
    // against 24.6 us; 128 x 4096 x 4096 the other way: 19.6 against 16.4).
    const long long tiles = static_cast<long long>(ceil_div(a.rows, kTmRows)) * p.nf;
    const bool worth = !dense || (4 * tiles <= num_sms && p.nk >= 32) || (2 * tiles <= num_sms && p.nk >= 64);
    p.ksplit_max = split && worth ? std::min(a.ksplit_max, kSplitSlicesMax) : 1;
    p.part = reinterpret_cast<float*>(a.part);
    p.part_rows = a.rows;
    p.tickets = a.tickets;
    p.ticket_cap = a.ticket_cap;
    // persistent: one CTA (or pair) per SM, fewer when the units cannot fill them
    const int tile_rows = pair ? CfgPair::kPairRows : swap ? kSwapRows : kTmRows;
    const long long max_tiles = (static_cast<long long>(ceil_div(a.rows, tile_rows)) +
                                 std::min(p.G, a.rows)) * p.nf * p.ksplit_max;
    const int ctas = pair ? 2 * static_cast<int>(std::min<long long>(max_tiles, num_sms / 2))
                          : static_cast<int>(std::min<long long>(max_tiles, num_sms));
    if (swap) return gate_up ? launch_swap<true>(mw, ma, p, ctas, s, pdl)
                             : launch_swap<false>(mw, ma, p, ctas, s, pdl);
    return gate_up ? launch_one<true>(mw, ma, p, pair, wn, ctas, s, pdl)
                   : launch_one<false>(mw, ma, p, pair, wn, ctas, s, pdl);
}

}  // namespace moe
