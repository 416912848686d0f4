// grouped_gemm.cu -- grouped SwiGLU expert GEMMs on tcgen05 tensor cores.
//
// "MoE" (llm.rainlin.net), section 3: E_e(x) = W_down (SiLU(W_gate x) (.) W_up x), the
// gate_up weight of an expert is one [2f, D] matrix (gate rows, then up rows); section
// 3.2: the routed output is scaled by the routing weight and index-added back to its
// token.  "MoE 到底省了什么" (clxhxhhr.top), section 3: with few rows per expert the
// layer is bound by reading the expert weights, with many rows it is bound by compute.
//
// Three persistent, warp-specialised kernels share one structure: warp 0 fills a ring of
// shared-memory stages (TMA, 128-byte swizzle, 64-deep K steps), warp 1 owns the tensor
// memory and one of its threads issues tcgen05.mma (bf16 in, fp32 accumulate), and the
// epilogue warps drain a double-buffered TMEM accumulator with tcgen05.ld while the next
// tile accumulates.  Epilogues: h = SiLU(g) * u -> bf16 for gate_up; w * v -> fp32
// reductions into the token's output row (and/or fp32 y_sorted) for down.  The work list
// (group, feature block, row block) is derived on the device from the group offsets, so no
// host synchronisation is needed, and every wait is bounded.
//   * grouped_gemm_kernel<BN, GATE_UP>, weights on M: 128 weight rows x BN token rows
//     (16..128), for groups of a handful of rows -- an expert with two rows still fills
//     the 128-lane tile.  gate_up keeps the gate block in accumulator columns [0, BN) and
//     the up block in [BN, 2BN) so one thread holds both halves of a feature.  Also the
//     router's logits GEMM (one dense group, the reduction split into partial planes).
//   * grouped_gemm_tm_kernel<GATE_UP>, tokens on M: 128 token rows x 256 weight rows (128
//     gate + 128 up features, or 256 output features), 8 epilogue warps; features lie
//     along the accumulator's columns, so h leaves as 16-byte stores and the down results
//     as 4-wide vector reductions.
//   * grouped_gemm_pair_kernel<GATE_UP>, CTA pairs: clusters of two with
//     tcgen05.mma.cta_group::2 over 256 token rows x 256 weight rows, each CTA loading its
//     own token rows and half of the weights (.cta_group::2 TMA, no multicast), commits
//     multicast to both CTAs' barriers; its token rows must be contiguous, so gate_up
//     reads an expert-ordered copy of x.
// The other two kernels gather gate_up's token rows themselves: the producer warp's lanes
// copy 16-byte chunks of x[token] with cp.async into the 128-byte swizzle the MMA
// descriptor expects, zero-filling rows past the group.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <unordered_map>

#include "grouped_gemm.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

cudaError_t get_encoder() {
    std::call_once(g_encode_once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode ? cudaSuccess : cudaErrorNotSupported;
}

// 2-D bf16 view [rows, cols] (cols contiguous), box [box_rows, 64], 128-byte swizzle.
cudaError_t encode_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols,
                       int box_rows) {
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * 2};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(kBK), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// encode_map through a per-process cache keyed by (base, rows, cols, box): a descriptor
// depends on nothing else, and a layer call would otherwise encode 4 to 8 of them on the
// host.  The cache is bounded (cleared when full).
cudaError_t make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, int box_rows) {
    struct Key {
        const void* base;
        uint64_t rows, cols;
        int box;
        bool operator==(const Key& o) const {
            return base == o.base && rows == o.rows && cols == o.cols && box == o.box;
        }
    };
    struct Hash {
        size_t operator()(const Key& k) const {
            size_t h = std::hash<const void*>()(k.base);
            h = h * 1000003u ^ std::hash<uint64_t>()(k.rows);
            h = h * 1000003u ^ std::hash<uint64_t>()(k.cols);
            return h * 1000003u ^ static_cast<size_t>(k.box);
        }
    };
    static std::mutex mu;
    static std::unordered_map<Key, CUtensorMap, Hash> cache;
    const Key key{base, rows, cols, box_rows};
    {
        std::lock_guard<std::mutex> lock(mu);
        auto it = cache.find(key);
        if (it != cache.end()) {
            *m = it->second;
            return cudaSuccess;
        }
    }
    const cudaError_t err = encode_map(m, base, rows, cols, box_rows);
    if (err != cudaSuccess) return err;
    std::lock_guard<std::mutex> lock(mu);
    if (cache.size() >= 4096) cache.clear();
    cache.emplace(key, *m);
    return cudaSuccess;
}

template <int BN, bool GATE_UP>
cudaError_t launch_tpl(const CUtensorMap& mw, const CUtensorMap& ma, const Params& p, int grid,
                       cudaStream_t s, bool pdl) {
    using C = Cfg<BN, GATE_UP>;
    const size_t smem = 1024 + static_cast<size_t>(C::kStages) * C::kStageBytes +
                        (2 * C::kStages + 5) * 8 + 16 +
                        2 * (p.G + 1) * sizeof(int);
    auto kfn = grouped_gemm_kernel<BN, GATE_UP>;
    cudaError_t err = set_smem_limit(reinterpret_cast<const void*>(kfn), smem);
    if (err != cudaSuccess) return err;
    err = launch_kernel(kfn, dim3(grid), dim3(kThreads), smem, s, pdl, mw, ma, p);
    count_launches(1);
    return err;
}

template <bool GATE_UP>
cudaError_t launch_tm(const CUtensorMap& mw, const CUtensorMap& ma, const Params& p, int grid,
                      cudaStream_t s, bool pdl) {
    using C = CfgTm<>;
    const size_t smem = 1024 + static_cast<size_t>(C::kStages) * C::kStageBytes +
                        (2 * C::kStages + 5) * 8 + 16 + 2 * (p.G + 1) * sizeof(int) +
                        (GATE_UP ? 0 : kEpiStageBytes);
    auto kfn = grouped_gemm_tm_kernel<GATE_UP>;
    cudaError_t err = set_smem_limit(reinterpret_cast<const void*>(kfn), smem);
    if (err != cudaSuccess) return err;
    err = launch_kernel(kfn, dim3(grid), dim3(kTmThreads), smem, s, pdl, mw, ma, p);
    count_launches(1);
    return err;
}

template <bool GATE_UP>
cudaError_t launch_pair(const CUtensorMap& mw, const CUtensorMap& ma, const Params& p,
                        int npairs, cudaStream_t s, bool pdl) {
    using C = CfgPair;
    const size_t smem = 1024 + static_cast<size_t>(C::kStages) * C::kStageBytes +
                        (2 * C::kStages + 5) * 8 + 16 + 2 * (p.G + 1) * sizeof(int) +
                        (GATE_UP ? 0 : kEpiStageBytes);
    auto kfn = grouped_gemm_pair_kernel<GATE_UP>;
    cudaError_t err = set_smem_limit(reinterpret_cast<const void*>(kfn), smem);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * npairs);
    cfg.blockDim = dim3(kTmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    err = cudaLaunchKernelEx(&cfg, kfn, mw, ma, p);
    count_launches(1);
    return err;
}

}  // namespace

cudaError_t encode_tile_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols,
                            int box_rows) {
    const cudaError_t err = get_encoder();
    return err != cudaSuccess ? err : encode_map(m, base, rows, cols, box_rows);
}

int pick_block_rows(int rows, int groups) {
    const int avg = rows / (groups > 0 ? groups : 1);
    if (avg <= 16) return 16;
    if (avg <= 32) return 32;
    if (avg <= 64) return 64;
    return 128;
}

namespace {

enum class Kind { kSwap, kTm, kPair };

// One launch of one kernel kind over every group.  BN: largest rows per tile of the
// weights-on-M kernel.
cudaError_t launch_kind(const GroupedGemmLaunch& a, Kind kind, int BN, int num_sms,
                        cudaStream_t s, bool pdl) {
    const bool tm = kind != Kind::kSwap;
    const int K = a.gate_up ? a.D : a.f;
    const uint64_t w_group_rows = a.gate_up ? 2ull * a.f : static_cast<uint64_t>(a.D);
    CUtensorMap mw, ma;
    cudaError_t err;
    if ((err = make_map(&mw, a.w, w_group_rows * a.E, K, kBM)) != cudaSuccess) return err;  // 128-row boxes
    // the activation map is only read when the rows are contiguous (no gather); with a
    // gather it still has to be a valid descriptor, so it covers the first row of x
    const void* act = a.act;
    bool gather = a.gate_up && a.gather_tok != nullptr;
    if (kind == Kind::kPair && gather) {
        err = launch_gather_rows(reinterpret_cast<const bf16*>(a.act), a.gather_tok, a.rows, a.D,
                                 a.gather_buf, num_sms, s, pdl);
        if (err != cudaSuccess) return err;
        act = a.gather_buf;
        gather = false;
    }
    // activation boxes: 128 rows (tokens on M) or BN rows (weights on M: one box per stage)
    if ((err = make_map(&ma, act, gather ? 1 : a.rows, K, gather ? 1 : (tm ? kTmRows : BN))) !=
        cudaSuccess)
        return err;
    Params p{};
    p.offsets = a.offsets;
    p.rows_total = a.rows;
    p.sorted_token = a.sorted_token;
    p.sorted_w = a.sorted_w;
    p.G = a.E;
    p.nf = a.gate_up ? a.f / kBM : a.D / (tm ? kTmN : kBM);
    p.nk = K / kBK;
    p.w_group_rows = static_cast<int>(w_group_rows);
    p.up_rows = a.f;
    p.out_cols = a.gate_up ? a.f : a.D;
    p.h_out = a.h_out;
    p.acc_out = a.acc_out;
    p.y_out = a.y_out;
    p.y16_out = a.gate_up ? nullptr : a.y16_out;
    p.status = a.status;
    p.gather_tok = gather ? a.gather_tok : nullptr;
    p.x = reinterpret_cast<const bf16*>(act);
    p.final_out = (!a.gate_up && a.acc_out && a.done) ? a.final_out : nullptr;
    p.final_rows = a.final_rows;
    p.done = a.done;
    p.final_residual = a.final_residual;
    p.barrier_budget_ns = a.barrier_budget_ns;
    p.ksplit = kind == Kind::kSwap && a.ksplit > 1 ? a.ksplit : 1;
    p.zero_acc = a.gate_up ? a.zero_acc : nullptr;
    p.zero_n4 = a.zero_floats / 4;
    p.act_box = BN;
    p.split_stride = static_cast<long long>(a.rows) * p.out_cols;
    // K split chosen on the device: gate_up needs the partial-sum planes and tickets, down
    // adds its slices into the fp32 accumulator (not into per-row outputs)
    const bool auto_split =
        kind != Kind::kPair && p.ksplit == 1 && a.ksplit_max > 1 &&
        (a.gate_up ? (a.part != nullptr && a.tickets != nullptr && a.ticket_cap > 0)
                   : (a.acc_out != nullptr && a.y_out == nullptr && a.y16_out == nullptr));
    p.ksplit_max = auto_split ? std::min(a.ksplit_max, kSplitSlicesMax) : 1;
    p.part = a.part;
    p.part_rows = a.rows;
    p.tickets = a.tickets;
    p.ticket_cap = a.ticket_cap;
    // persistent grids: one CTA (or pair) per SM, fewer when the units cannot fill them
    const int rows_per_tile = kind == Kind::kPair ? CfgPair::kPairRows : (tm ? kTmRows : 16);
    const long long max_tiles = (static_cast<long long>(ceil_div(a.rows, rows_per_tile)) + p.G) *
                                p.nf * p.ksplit * p.ksplit_max;
    if (kind == Kind::kPair) {
        const int npairs = static_cast<int>(std::min<long long>(max_tiles, num_sms / 2));
        return a.gate_up ? launch_pair<true>(mw, ma, p, npairs, s, true)
                         : launch_pair<false>(mw, ma, p, npairs, s, true);
    }
    const int grid = static_cast<int>(max_tiles < num_sms ? max_tiles : num_sms);
    if (tm) return a.gate_up ? launch_tm<true>(mw, ma, p, grid, s, pdl)
                             : launch_tm<false>(mw, ma, p, grid, s, pdl);
    switch (BN) {
        case 16: return a.gate_up ? launch_tpl<16, true>(mw, ma, p, grid, s, pdl) : launch_tpl<16, false>(mw, ma, p, grid, s, pdl);
        case 32: return a.gate_up ? launch_tpl<32, true>(mw, ma, p, grid, s, pdl) : launch_tpl<32, false>(mw, ma, p, grid, s, pdl);
        case 64: return a.gate_up ? launch_tpl<64, true>(mw, ma, p, grid, s, pdl) : launch_tpl<64, false>(mw, ma, p, grid, s, pdl);
        case 128: return a.gate_up ? launch_tpl<128, true>(mw, ma, p, grid, s, pdl) : launch_tpl<128, false>(mw, ma, p, grid, s, pdl);
        // 256 token rows: down only (gate_up's two accumulators would not fit tensor memory)
        default: return a.gate_up ? cudaErrorInvalidValue : launch_tpl<256, false>(mw, ma, p, grid, s, pdl);
    }
}

}  // namespace

namespace {

// Kernel kind and weights-on-M tile height for a launch (see launch_grouped_gemm).
bool pick_kind(const GroupedGemmLaunch& a, int num_sms, Kind* kind, int* BN) {
    // tokens on M needs f (gate_up) or D (down) in 128- or 256-wide blocks
    const bool tm_ok = a.gate_up ? (a.f % 128 == 0) : (a.D % 256 == 0);
    const bool gathered = a.gate_up && a.gather_tok != nullptr;
    const bool pair_ok = tm_ok && (!gathered || a.gather_buf != nullptr) && num_sms >= 2;
    const int routed_rows = a.rows;
    // weights on M: tiles adapt per group up to BN, sized for groups up to 8x the average
    // (skewed routing) but never past the largest possible group
    const int max_rows = a.max_group_rows > 0 ? a.max_group_rows : routed_rows;
    const long long avg8 = 8ll * routed_rows / a.E;
    const int bn_rows = static_cast<int>(std::min<long long>(max_rows, std::max(avg8, 16ll)));
    *BN = a.block_rows ? a.block_rows : pick_block_rows(bn_rows, 1);
    if (*BN != 16 && *BN != 32 && *BN != 64 && *BN != 128 && !(*BN == 256 && !a.gate_up))
        return false;
    if (a.ksplit > 1 && (a.gate_up || !a.y_out || a.acc_out || a.final_out ||
                         (a.f / kBK) % a.ksplit != 0))
        return false;
    // Orientation.  Weights on M (token tiles of 16..128 rows) when asked for (the router's
    // split-reduction logits GEMM), or when the tokens-on-M tiles do not divide the shape.
    // Otherwise tokens on M: both orientations stream each weight tile once per row block
    // and are within a few percent of each other on 2-row groups, but tokens on M keeps
    // features along the accumulator's columns (16-byte stores and vector reductions in
    // the epilogue) and wins clearly once groups hold tens of rows; when a few experts (a
    // handful of tokens, or concentrated routing) give fewer tiles than the grid has CTAs,
    // both cut each tile's K steps on the device.  CTA pairs once the groups
    // average a full 256-row pair tile's half (their rows must be contiguous: x is
    // gathered first).
    if (a.orientation == 1 || a.block_rows || !tm_ok || a.ksplit > 1)
        *kind = Kind::kSwap;
    else if (a.orientation == 2)
        *kind = Kind::kTm;
    else if (a.orientation == 3 || routed_rows / a.E >= 128)
        *kind = pair_ok ? Kind::kPair : Kind::kTm;
    else
        *kind = max_rows <= kSwapMaxRows ? Kind::kSwap : Kind::kTm;
    return true;
}

}  // namespace

int grouped_gemm_launches(const GroupedGemmLaunch& a, int num_sms) {
    Kind kind;
    int BN;
    if (a.rows == 0 || a.E == 0 || !pick_kind(a, num_sms, &kind, &BN)) return 0;
    return (kind == Kind::kPair && a.gate_up && a.gather_tok != nullptr) ? 2 : 1;
}

bool grouped_gemm_uses_pairs(const GroupedGemmLaunch& a, int num_sms) {
    Kind kind;
    int BN;
    return pick_kind(a, num_sms, &kind, &BN) && kind == Kind::kPair;
}


cudaError_t launch_grouped_gemm(const GroupedGemmLaunch& a, int num_sms, cudaStream_t s,
                                bool pdl) {
    if (a.rows == 0 || a.E == 0) return cudaSuccess;
    if (a.E > kMaxGroups) return cudaErrorInvalidValue;
    cudaError_t err = get_encoder();
    if (err != cudaSuccess) return err;
    Kind kind;
    int BN;
    if (!pick_kind(a, num_sms, &kind, &BN)) return cudaErrorInvalidValue;
    return launch_kind(a, kind, BN, num_sms, s, pdl);
}

}  // namespace moe
