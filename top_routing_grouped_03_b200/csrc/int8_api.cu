// int8_api.cu -- the extern "C" entry points of routing by a rule and of the layer in 8-bit
// integers: argument checks on the host, workspace layout, launch sequences.  See
// include/moe_api.h.
#include <algorithm>
#include <cmath>

#include "api_util.cuh"

namespace moe {
namespace {

struct Taker {
    size_t end = 0;
    size_t operator()(size_t bytes) {
        const size_t r = end;
        end = align_up(end + bytes);
        return r;
    }
};

int check_rule(const moe_route_rule* r, int E, int K) {
    if (!r) return MOE_ERR_ARG;
    if (r->score_mode != MOE_SCORE_SOFTMAX && r->score_mode != MOE_SCORE_SIGMOID) return MOE_ERR_ARG;
    if (r->n_group < 1 || E % r->n_group || r->topk_group < 1 || r->topk_group > r->n_group)
        return MOE_ERR_ARG;
    if (r->n_group > 32) return MOE_ERR_UNSUPPORTED;
    if (r->topk_group * (E / r->n_group) < K) return MOE_ERR_ARG;
    if ((r->group_top != 1 && r->group_top != 2) || !std::isfinite(r->scale)) return MOE_ERR_ARG;
    return MOE_OK;
}

RouteLogitsLaunch rule_launch(const moe_route_rule* r) {
    RouteLogitsLaunch a{};
    a.planes = 1;
    a.score_mode = r->score_mode;
    a.select_bias = r->select_bias;
    a.n_group = r->n_group;
    a.topk_group = r->topk_group;
    a.group_top = r->group_top;
    a.renorm = r->renorm ? 1 : 0;
    a.scale = r->scale;
    return a;
}

// A rule in the place of p's own routing.
int check_layer_rule(const moe_layer_params* p, const moe_route_rule* rule) {
    int rc = check_shape(p->T, p->D, p->E, p->K, p->f, p->f_s);
    if (rc) return rc;
    if ((rc = check_rule(rule, p->E, p->K))) return rc;
    return p->score_mode || p->select_bias || (p->flags & MOE_FLAG_BF16_WEIGHTS) ? MOE_ERR_ARG : MOE_OK;
}

// ---------------------------------------------------------------- dense product

// The K steps of a tile may be cut into slices when the tiles cannot fill the GPU; the slices'
// int32 planes of [T, N] meet in the workspace if they take at most 64 MiB.
constexpr int kDenseTileN = 64;  // the narrowest tile: the most tickets
long long dense_tiles(long long T, long long N) {
    return ((T + 127) / 128) * ((N + kDenseTileN - 1) / kDenseTileN);
}
bool dense_split_ok(long long T, long long N) { return 4ll * kSplitMax * T * N <= (64ll << 20) && dense_tiles(T, N) < 4 * 296; }

struct DenseLayout {
    size_t status, tickets, part, xq, xs, total;
    int ticket_cap, clear_words;
};
DenseLayout dense_layout(long long T, long long N, long long K) {
    DenseLayout L{};
    Taker take;
    const bool split = dense_split_ok(T, N);
    L.ticket_cap = split ? static_cast<int>(dense_tiles(T, N)) : 0;
    L.status = take(kAlign);
    L.tickets = take(sizeof(unsigned) * L.ticket_cap);
    L.clear_words = static_cast<int>(take.end / 4);
    L.part = take(split ? 4ull * kSplitMax * T * N : 0);
    L.xq = take(T * K);
    L.xs = take(sizeof(float) * T);
    L.total = take.end;
    return L;
}

int check_dense(int T, int N, int K) {
    if (T < 0 || N <= 0 || K <= 0) return MOE_ERR_ARG;
    if (N % 8 || N > (1 << 20) || K % 16 || K > 65536) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

cudaError_t launch_dense(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws_, int T,
                         int N, int K, moe_bf16* out, void* workspace, const DenseLayout& L,
                         cudaStream_t s, bool pdl) {
    Int8GemmLaunch g{};
    g.kind = Int8GemmLaunch::kDense;
    g.w = wq;
    g.w_scale = ws_;
    g.act = xq;
    g.act_scale = xs;
    g.rows = g.tokens = T;
    g.E = 1;
    g.D = N;
    g.f = K;
    g.y16_out = reinterpret_cast<bf16*>(out);
    g.status = at<int>(workspace, L.status);
    if (L.ticket_cap > 0) {
        g.ksplit_max = kSplitMax;
        g.part = at<void>(workspace, L.part);
        g.tickets = at<unsigned>(workspace, L.tickets);
        g.ticket_cap = L.ticket_cap;
    }
    return launch_int8_gemm(g, num_sms_current(), s, pdl);
}

// ---------------------------------------------------------------- experts

struct ExpertsLayout {
    size_t status, tickets, gather, h, hq, hs, acc, y, y_scale, part, total;
    size_t zero_end;
};
void take_experts(Taker& take, ExpertsLayout& L, long long T, long long D, long long E, long long K,
                  long long f, unsigned flags) {
    const long long rows = T * K;
    const bool det = (flags & MOE_FLAG_DETERMINISTIC) != 0, pairs = rows / E >= 128;
    L.gather = take(pairs ? rows * D : 0);
    L.h = take(sizeof(float) * rows * f);
    L.hq = take(rows * f);
    L.hs = take(sizeof(float) * rows);
    L.acc = take(sizeof(float) * T * D);
    // rows for a sum by the combine: fp32 (fixed order), 16-bit integers and scales (CTA pairs)
    L.y = take(det ? sizeof(float) * rows * D : pairs ? sizeof(int16_t) * rows * D : 0);
    L.y_scale = take(!det && pairs ? sizeof(float) * rows * (D / 32) : 0);
    L.part = take(gate_up_split_ok(T, K, f) ? sizeof(float) * kSplitMax * rows * 2 * f : 0);
}
ExpertsLayout experts_layout(long long T, long long D, long long E, long long K, long long f,
                             unsigned flags) {
    ExpertsLayout L{};
    Taker take;
    L.status = take(kAlign);
    L.tickets = take(sizeof(unsigned) * gate_up_ticket_cap(T, E, K, f));
    L.zero_end = take.end;
    take_experts(take, L, T, D, E, K, f, flags);
    L.total = take.end;
    return L;
}

// How the rows of a token's experts are summed: in the fp32 accumulator by reductions, or from
// their rows in memory by the combine (unweighted fp32 rows in slot order; on CTA pairs, where
// reductions would hold up the tensor cores, weighted 16-bit rows).
enum class Sum { kAccumulator, kRows, kRows16 };

// gate_up, the quantised h and down of the routed experts.  acc (or NULL) is zeroed on the way.
cudaError_t run_experts(const moe_int8_experts& p, const ExpertsLayout& L, void* ws, Sum sum, float* acc,
                        int sms, cudaStream_t s, bool pdl) {
    const int rows = p.T * p.K;
    Int8GemmLaunch up{};
    up.kind = Int8GemmLaunch::kGateUp;
    up.w = p.w_gate_up;
    up.w_scale = p.gate_up_scale;
    up.act = p.xq;
    up.act_scale = p.x_scale;
    up.offsets = p.expert_offsets;
    up.sorted_token = p.sorted_token;
    up.rows = rows; up.tokens = p.T; up.E = p.E; up.D = p.D; up.f = p.f;
    up.h_out = at<float>(ws, L.h);
    up.status = at<int>(ws, L.status);
    up.gather_buf = rows / p.E >= 128 ? at<int8_t>(ws, L.gather) : nullptr;
    if (acc) {
        up.zero_acc = acc;
        up.zero_floats = static_cast<long long>(p.T) * p.D;
    }
    if (gate_up_split_ok(p.T, p.K, p.f)) {
        up.ksplit_max = kSplitMax;
        up.part = at<void>(ws, L.part);
        up.tickets = at<unsigned>(ws, L.tickets);
        up.ticket_cap = static_cast<int>(gate_up_ticket_cap(p.T, p.E, p.K, p.f));
    }
    cudaError_t err = launch_int8_gemm(up, sms, s, pdl);
    if (err != cudaSuccess) return err;
    QuantizeLaunch q{};
    q.x = up.h_out;
    q.is_f32 = true;
    q.rows = rows;
    q.cols = p.f;
    q.q = at<int8_t>(ws, L.hq);
    q.scale = at<float>(ws, L.hs);
    q.row_count = p.expert_offsets + p.E;
    if ((err = launch_quantize(q, s, true)) != cudaSuccess) return err;
    Int8GemmLaunch dn{};
    dn.kind = Int8GemmLaunch::kDown;
    dn.w = p.w_down;
    dn.w_scale = p.down_scale;
    dn.act = q.q;
    dn.act_scale = q.scale;
    dn.offsets = p.expert_offsets;
    dn.sorted_token = p.sorted_token;
    dn.sorted_w = sum == Sum::kRows ? nullptr : p.sorted_w;
    dn.rows = rows; dn.tokens = p.T; dn.E = p.E; dn.D = p.D; dn.f = p.f;
    if (sum == Sum::kAccumulator) dn.acc_out = acc;
    if (sum == Sum::kRows) dn.y_out = at<float>(ws, L.y);
    if (sum == Sum::kRows16) {
        dn.y16q_out = at<int16_t>(ws, L.y);
        dn.y16q_scale = at<float>(ws, L.y_scale);
    }
    dn.status = up.status;
    dn.ksplit_max = sum == Sum::kAccumulator ? kSplitMax : 1;
    return launch_int8_gemm(dn, sms, s, true);
}

Sum pick_sum(int T, int D, int E, int K, int f, unsigned flags, int sms) {
    if (flags & MOE_FLAG_DETERMINISTIC) return Sum::kRows;
    Int8GemmLaunch dn{};
    dn.kind = Int8GemmLaunch::kDown;
    dn.rows = T * K; dn.tokens = T; dn.E = E; dn.D = D; dn.f = f;
    return T * K / E >= 128 && int8_gemm_uses_pairs(dn, sms) ? Sum::kRows16 : Sum::kAccumulator;
}

// The end of a call: the accumulator (or NULL), the rows and the residual to out.
cudaError_t run_combine(const ExpertsLayout& L, void* ws, Sum sum, const float* acc,
                        const int32_t* slot_to_row, const float* topk_w, const moe_bf16* residual, int T,
                        int D, int K, moe_bf16* out, int sms, cudaStream_t s) {
    CombineLaunch c{};
    c.residual = reinterpret_cast<const bf16*>(residual);
    c.out_acc = acc;
    c.slot_to_row = slot_to_row;
    if (sum == Sum::kRows) {
        c.y_sorted = at<float>(ws, L.y);
        c.topk_w = topk_w;
    }
    if (sum == Sum::kRows16) {
        c.y16q_sorted = at<int16_t>(ws, L.y);
        c.y16q_scale = at<float>(ws, L.y_scale);
    }
    c.T = T; c.D = D; c.K = K;
    c.out = reinterpret_cast<bf16*>(out);
    return launch_combine(c, sms, s, true);
}

// The whole of moe_experts_int8 for a handful of rows: three launches.  status: the status word to
// clear, NULL in a layer call (which has cleared it, and whose permutation may have set it).
cudaError_t run_few(const moe_int8_experts& p, const ExpertsLayout& L, void* ws, int* status, moe_bf16* out,
                    int sms, cudaStream_t s) {
    Int8FewExperts a{};
    a.xq = p.xq;
    a.x_scale = p.x_scale;
    a.offsets = p.expert_offsets;
    a.sorted_token = p.sorted_token;
    a.sorted_w = p.sorted_w;
    a.w_gate_up = p.w_gate_up;
    a.gate_up_scale = p.gate_up_scale;
    a.w_down = p.w_down;
    a.down_scale = p.down_scale;
    a.residual = reinterpret_cast<const bf16*>(p.residual);
    a.T = p.T; a.D = p.D; a.E = p.E; a.K = p.K; a.f = p.f;
    a.h = at<float>(ws, L.h);
    a.hq = at<int8_t>(ws, L.hq);
    a.hs = at<float>(ws, L.hs);
    a.status = status;
    a.out = reinterpret_cast<bf16*>(out);
    return launch_few_experts(a, sms, s);
}

int check_experts_shape(int T, int D, int E, int K, int f) {
    const int rc = check_shape(T, D, E, K, f, 0);
    if (rc) return rc;
    // the gather's offsets count pairs of bytes in 32 bits
    return static_cast<long long>(T) * D >= (1ll << 33) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// ---------------------------------------------------------------- layer

struct LayerLayout {
    ExpertsLayout x;
    size_t counters, counts, perm_hist, logits, offsets, topk_idx, topk_w, sgate, sorted_token, sorted_w,
        slot_to_row, xq, xs, h_s, hq_s, hs_s, total;
};
LayerLayout layer_layout(long long T, long long D, long long E, long long K, long long f,
                         long long fs, unsigned flags) {
    LayerLayout L{};
    Taker take;
    L.x.status = take(kAlign);
    L.counters = take(sizeof(unsigned) * ((T + 7) / 8));
    L.counts = take(sizeof(int32_t) * E);
    L.x.tickets = take(sizeof(unsigned) * gate_up_ticket_cap(T, E, K, f));
    L.x.zero_end = take.end;
    L.perm_hist = take(sizeof(int32_t) * E * permute_chunks(T * K));
    const bool tc = router_uses_tensor_cores(static_cast<int>(T), static_cast<int>(E));
    L.logits = take(sizeof(float) * T *
                    std::max<long long>(E + 1, tc ? router_tc_max_planes(static_cast<int>(T)) * E : 0));
    L.offsets = take(sizeof(int32_t) * (E + 1));
    L.topk_idx = take(sizeof(int32_t) * T * K);
    L.topk_w = take(sizeof(float) * T * K);
    L.sgate = take(sizeof(float) * T);
    L.sorted_token = take(sizeof(int32_t) * T * K);
    L.sorted_w = take(sizeof(float) * T * K);
    L.slot_to_row = take(sizeof(int32_t) * T * K);
    L.xq = take(T * D);
    L.xs = take(sizeof(float) * T);
    L.h_s = take(sizeof(float) * T * fs);
    L.hq_s = take(T * fs);
    L.hs_s = take(fs ? sizeof(float) * T : 0);
    take_experts(take, L.x, T, D, E, K, f, flags);
    L.total = take.end;
    return L;
}

int layer_int8(const moe_layer_params* p, const RouteLogitsLaunch* rule, const moe_int8_weights* w,
               moe_bf16* out, void* ws, size_t ws_bytes, cudaStream_t s) {
    const int T = p->T, D = p->D, E = p->E, K = p->K, f = p->f, fs = p->f_s;
    int rc = check_shape(T, D, E, K, f, fs);
    if (rc) return rc;
    if (static_cast<long long>(T) * D >= (1ll << 33)) return MOE_ERR_UNSUPPORTED;
    const bool shared = fs > 0;
    if (!p->w_router || p->w_gate_up || p->w_down || p->w_shared_gate_up || p->w_shared_down ||
        p->step_events)
        return MOE_ERR_ARG;
    if (!w->gate_up || !w->gate_up_scale || !w->down || !w->down_scale) return MOE_ERR_ARG;
    const bool any = p->w_shared_gate || w->shared_gate_up || w->shared_gate_up_scale || w->shared_down ||
                     w->shared_down_scale;
    const bool all = p->w_shared_gate && w->shared_gate_up && w->shared_gate_up_scale &&
                     w->shared_down && w->shared_down_scale;
    if (shared ? !all : any) return MOE_ERR_ARG;
    if (p->score_mode != MOE_SCORE_SOFTMAX && p->score_mode != MOE_SCORE_SIGMOID) return MOE_ERR_ARG;
    if (!(p->capacity_factor >= 0.f) || !std::isfinite(p->capacity_factor) || p->min_capacity < 0)
        return MOE_ERR_ARG;
    const void* ptrs[] = {p->x, p->w_router, p->w_shared_gate, p->residual, out, w->gate_up,
                          w->gate_up_scale, w->down, w->down_scale, w->shared_gate_up,
                          w->shared_gate_up_scale, w->shared_down, w->shared_down_scale};
    for (const void* q : ptrs)
        if (!aligned16(q)) return MOE_ERR_ALIGN;
    if (T > 0 && (!p->x || !out)) return MOE_ERR_ARG;
    if (!ws) return MOE_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return MOE_ERR_ALIGN;
    const LayerLayout L = layer_layout(T, D, E, K, f, fs, p->flags);
    if (ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    if (T == 0) return MOE_OK;
    const int sms = num_sms_current();
    const bool det = (p->flags & MOE_FLAG_DETERMINISTIC) != 0;
    int* status = at<int>(ws, L.x.status);
    if (cudaMemsetAsync(ws, 0, L.x.zero_end, s) != cudaSuccess) return MOE_ERR_CUDA;

    const bool tc = router_uses_tensor_cores(T, E);
    RouterLaunch r{};
    r.x = reinterpret_cast<const bf16*>(p->x);
    r.w_router = reinterpret_cast<const bf16*>(p->w_router);
    r.logit_bias = p->logit_bias;
    r.w_shared_gate = reinterpret_cast<const bf16*>(p->w_shared_gate);
    r.T = T; r.D = D; r.E = E; r.K = K;
    r.logits = at<float>(ws, L.logits);
    r.counters = at<unsigned>(ws, L.counters);
    r.topk_idx = p->topk_idx_out ? p->topk_idx_out : at<int32_t>(ws, L.topk_idx);
    r.topk_w = p->topk_w_out ? p->topk_w_out : at<float>(ws, L.topk_w);
    r.counts = tc ? nullptr : at<int32_t>(ws, L.counts);
    r.shared_gate = at<float>(ws, L.sgate);
    r.status = status;
    r.score_mode = p->score_mode;
    r.select_bias = p->select_bias;
    r.bf16_weights = (p->flags & MOE_FLAG_BF16_WEIGHTS) ? 1 : 0;
    r.rule = rule;
    if ((tc ? launch_router_tc(r, sms, s) : launch_router(r, sms, s)) != cudaSuccess)
        return MOE_ERR_CUDA;
    QuantizeLaunch q{};
    q.x = p->x;
    q.rows = T;
    q.cols = D;
    q.q = at<int8_t>(ws, L.xq);
    q.scale = at<float>(ws, L.xs);
    if (launch_quantize(q, s, true) != cudaSuccess) return MOE_ERR_CUDA;
    PermuteLaunch pm{};
    pm.topk_idx = r.topk_idx;
    pm.topk_w = r.topk_w;
    pm.counts = r.counts;
    pm.counts_out = p->expert_counts_out;
    pm.T = T; pm.E = E; pm.K = K;
    pm.offsets = at<int32_t>(ws, L.offsets);
    pm.sorted_token = at<int32_t>(ws, L.sorted_token);
    pm.sorted_w = at<float>(ws, L.sorted_w);
    pm.slot_to_row = at<int32_t>(ws, L.slot_to_row);
    pm.status = status;
    pm.hist = at<int32_t>(ws, L.perm_hist);
    pm.capacity = p->capacity_factor > 0.f
                      ? moe_expert_capacity(T, K, E, p->capacity_factor, p->min_capacity)
                      : -1;
    if (launch_permute(pm, s, true) != cudaSuccess) return MOE_ERR_CUDA;

    moe_int8_experts e{};
    e.xq = q.q;
    e.x_scale = q.scale;
    e.expert_offsets = pm.offsets;
    e.sorted_token = pm.sorted_token;
    e.sorted_w = pm.sorted_w;
    e.w_gate_up = w->gate_up;
    e.gate_up_scale = w->gate_up_scale;
    e.w_down = w->down;
    e.down_scale = w->down_scale;
    e.residual = p->residual;
    e.T = T; e.D = D; e.E = E; e.K = K; e.f = f;
    if (!shared && few_experts_ok(T, D, K, f))
        return run_few(e, L.x, ws, nullptr, out, sms, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    const Sum sum = pick_sum(T, D, E, K, f, p->flags, sms);
    // the accumulator: the routed rows' reductions and the shared expert's
    float* acc = sum == Sum::kAccumulator || shared ? at<float>(ws, L.x.acc) : nullptr;
    if (run_experts(e, L.x, ws, sum, acc, sms, s, true) != cudaSuccess) return MOE_ERR_CUDA;
    if (shared) {
        Int8GemmLaunch su{};
        su.kind = Int8GemmLaunch::kGateUp;
        su.w = w->shared_gate_up;
        su.w_scale = w->shared_gate_up_scale;
        su.act = q.q;
        su.act_scale = q.scale;
        su.rows = su.tokens = T;
        su.E = 1; su.D = D; su.f = fs;
        su.h_out = at<float>(ws, L.h_s);
        su.status = status;
        if (launch_int8_gemm(su, sms, s, true) != cudaSuccess) return MOE_ERR_CUDA;
        QuantizeLaunch qs{};
        qs.x = su.h_out;
        qs.is_f32 = true;
        qs.rows = T;
        qs.cols = fs;
        qs.q = at<int8_t>(ws, L.hq_s);
        qs.scale = at<float>(ws, L.hs_s);
        if (launch_quantize(qs, s, true) != cudaSuccess) return MOE_ERR_CUDA;
        Int8GemmLaunch sd{};
        sd.kind = Int8GemmLaunch::kDown;
        sd.w = w->shared_down;
        sd.w_scale = w->shared_down_scale;
        sd.act = qs.q;
        sd.act_scale = qs.scale;
        sd.sorted_w = r.shared_gate;
        sd.rows = sd.tokens = T;
        sd.E = 1; sd.D = D; sd.f = fs;
        sd.acc_out = acc;
        sd.status = status;
        sd.ksplit_max = det ? 1 : kSplitMax;
        if (launch_int8_gemm(sd, sms, s, true) != cudaSuccess) return MOE_ERR_CUDA;
    }
    return run_combine(L.x, ws, sum, acc, pm.slot_to_row, r.topk_w, p->residual, T, D, K, out, sms, s) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_route_logits(const void* logits, int logits_dtype, int T, int E, int K,
                     const moe_route_rule* rule, int32_t* topk_idx, float* topk_w,
                     int32_t* expert_counts, void* stream) {
    int rc = check_shape(T, 128, E, K, 128, 0);
    if (rc) return rc;
    if ((rc = check_rule(rule, E, K))) return rc;
    if (logits_dtype != MOE_DTYPE_F32 && logits_dtype != MOE_DTYPE_BF16) return MOE_ERR_ARG;
    if (T > 0 && (!logits || !topk_idx || !topk_w)) return MOE_ERR_ARG;
    RouteLogitsLaunch a = rule_launch(rule);
    a.logits = logits;
    a.is_bf16 = logits_dtype == MOE_DTYPE_BF16;
    a.row_stride = E;
    a.T = T; a.E = E; a.K = K;
    a.topk_idx = topk_idx;
    a.topk_w = topk_w;
    a.counts = expert_counts;
    return launch_route_logits(a, num_sms_current(), as_stream(stream)) == cudaSuccess ? MOE_OK
                                                                                        : MOE_ERR_CUDA;
}

int moe_route_rule_ex(const moe_bf16* x, const moe_bf16* w_router, const float* logit_bias,
                      const moe_bf16* w_shared_gate, int T, int D, int E, int K,
                      const moe_route_rule* rule, int32_t* topk_idx, float* topk_w,
                      int32_t* expert_counts, float* shared_gate, void* workspace, size_t ws_bytes,
                      void* stream) {
    int rc = check_shape(T, D, E, K, 128, 0);
    if (rc) return rc;
    if ((rc = check_rule(rule, E, K))) return rc;
    if (!w_router || !expert_counts) return MOE_ERR_ARG;
    if (T > 0 && (!x || !topk_idx || !topk_w || (w_shared_gate && !shared_gate))) return MOE_ERR_ARG;
    if (!aligned16(x) || !aligned16(w_router) || !aligned16(w_shared_gate)) return MOE_ERR_ALIGN;
    if (!workspace || ws_bytes < moe_workspace_size(T, D, E, K, 128, 0)) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOE_ERR_ALIGN;  // the logits are stored in vectors
    cudaStream_t s = as_stream(stream);
    const RouteLogitsLaunch rl = rule_launch(rule);
    if (T == 0)
        return cudaMemsetAsync(expert_counts, 0, sizeof(int32_t) * E, s) == cudaSuccess ? MOE_OK
                                                                                        : MOE_ERR_CUDA;
    if (cudaMemsetAsync(workspace, 0, kAlign, s) != cudaSuccess) return MOE_ERR_CUDA;  // the status word
    RouterLaunch a{};
    a.x = reinterpret_cast<const bf16*>(x);
    a.w_router = reinterpret_cast<const bf16*>(w_router);
    a.logit_bias = logit_bias;
    a.w_shared_gate = reinterpret_cast<const bf16*>(w_shared_gate);
    a.T = T; a.D = D; a.E = E; a.K = K;
    a.logits = at<float>(workspace, kAlign);
    a.topk_idx = topk_idx;
    a.topk_w = topk_w;
    a.counts = expert_counts;
    a.shared_gate = shared_gate;
    a.status = at<int>(workspace, 0);
    a.rule = &rl;
    const int sms = num_sms_current();
    const cudaError_t err = router_uses_tensor_cores(T, E) ? launch_router_tc(a, sms, s)
                                                           : launch_router(a, sms, s);
    return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_quantize_rows(const moe_bf16* x, long long rows, int cols, int8_t* q, float* scale,
                      void* stream) {
    if (rows < 0 || cols <= 0) return MOE_ERR_ARG;
    if (cols % 16 || rows >= (1ll << 31)) return MOE_ERR_UNSUPPORTED;
    if (rows > 0 && (!x || !q || !scale)) return MOE_ERR_ARG;
    if (!aligned16(x) || !aligned16(q)) return MOE_ERR_ALIGN;
    QuantizeLaunch a{};
    a.x = x;
    a.rows = rows;
    a.cols = cols;
    a.q = q;
    a.scale = scale;
    return launch_quantize(a, as_stream(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_int8_workspace_size(int T, int N, int K) {
    // a handful of tokens needs none
    return check_dense(T, N, K) != MOE_OK || few_linear_ok(T, K) ? 0 : dense_layout(T, N, K).total;
}

int moe_int8_matmul(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
                    int T, int N, int K, moe_bf16* out, void* workspace, size_t ws_bytes,
                    void* stream) {
    const int rc = check_dense(T, N, K);
    if (rc) return rc;
    if (!wq || !w_scale || (T > 0 && (!xq || !x_scale || !out))) return MOE_ERR_ARG;
    if (!aligned16(xq) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(out)) return MOE_ERR_ALIGN;
    if (T == 0) return MOE_OK;
    cudaStream_t s = as_stream(stream);
    if (few_linear_ok(T, K))
        return launch_few_linear(nullptr, xq, x_scale, wq, w_scale, T, N, K,
                                 reinterpret_cast<bf16*>(out), num_sms_current(), s) == cudaSuccess
                   ? MOE_OK
                   : MOE_ERR_CUDA;
    const DenseLayout L = dense_layout(T, N, K);
    if (!workspace || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0) return MOE_ERR_ALIGN;
    if (cudaMemsetAsync(workspace, 0, 4ull * L.clear_words, s) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_dense(xq, x_scale, wq, w_scale, T, N, K, out, workspace, L, s, false) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

int moe_int8_linear(const moe_bf16* x, const int8_t* wq, const float* w_scale, int T, int N, int K,
                    moe_bf16* out, void* workspace, size_t ws_bytes, void* stream) {
    const int rc = check_dense(T, N, K);
    if (rc) return rc;
    if (!wq || !w_scale || (T > 0 && (!x || !out))) return MOE_ERR_ARG;
    if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(out)) return MOE_ERR_ALIGN;
    if (T == 0) return MOE_OK;
    cudaStream_t s = as_stream(stream);
    if (few_linear_ok(T, K))
        return launch_few_linear(reinterpret_cast<const bf16*>(x), nullptr, nullptr, wq, w_scale, T, N,
                                 K, reinterpret_cast<bf16*>(out), num_sms_current(), s) == cudaSuccess
                   ? MOE_OK
                   : MOE_ERR_CUDA;
    const DenseLayout L = dense_layout(T, N, K);
    if (!workspace || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0) return MOE_ERR_ALIGN;
    QuantizeLaunch q{};
    q.x = x;
    q.rows = T;
    q.cols = K;
    q.q = at<int8_t>(workspace, L.xq);
    q.scale = at<float>(workspace, L.xs);
    q.clear = at<unsigned>(workspace, 0);
    q.clear_words = L.clear_words;
    if (launch_quantize(q, s) != cudaSuccess) return MOE_ERR_CUDA;
    return launch_dense(q.q, q.scale, wq, w_scale, T, N, K, out, workspace, L, s, true) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

size_t moe_experts_int8_workspace_size(int T, int D, int E, int K, int f, unsigned flags) {
    return check_experts_shape(T, D, E, K, f) == MOE_OK ? experts_layout(T, D, E, K, f, flags).total : 0;
}

int moe_experts_int8(const moe_int8_experts* p, moe_bf16* out, void* workspace, size_t ws_bytes,
                     void* stream) {
    if (!p) return MOE_ERR_ARG;
    const int T = p->T, D = p->D, E = p->E, K = p->K, f = p->f;
    const int rc = check_experts_shape(T, D, E, K, f);
    if (rc) return rc;
    const bool det = (p->flags & MOE_FLAG_DETERMINISTIC) != 0;
    if (!p->expert_offsets || !p->w_gate_up || !p->gate_up_scale || !p->w_down || !p->down_scale)
        return MOE_ERR_ARG;
    if (T > 0 && (!p->xq || !p->x_scale || !p->sorted_token || !p->sorted_w || !out)) return MOE_ERR_ARG;
    if (T > 0 && (!p->slot_to_row || (det && !p->topk_w))) return MOE_ERR_ARG;
    const void* ptrs[] = {p->xq, p->w_gate_up, p->gate_up_scale, p->w_down, p->down_scale, p->residual, out};
    for (const void* q : ptrs)
        if (!aligned16(q)) return MOE_ERR_ALIGN;
    const ExpertsLayout L = experts_layout(T, D, E, K, f, p->flags);
    if (!workspace || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0) return MOE_ERR_ALIGN;
    if (T == 0) return MOE_OK;
    cudaStream_t s = as_stream(stream);
    const int sms = num_sms_current();
    if (few_experts_ok(T, D, K, f))
        return run_few(*p, L, workspace, at<int>(workspace, L.status), out, sms, s) == cudaSuccess ? MOE_OK
                                                                                                   : MOE_ERR_CUDA;
    if (cudaMemsetAsync(workspace, 0, L.zero_end, s) != cudaSuccess) return MOE_ERR_CUDA;
    const Sum sum = pick_sum(T, D, E, K, f, p->flags, sms);
    float* acc = sum == Sum::kAccumulator ? at<float>(workspace, L.acc) : nullptr;
    if (run_experts(*p, L, workspace, sum, acc, sms, s, false) != cudaSuccess) return MOE_ERR_CUDA;
    return run_combine(L, workspace, sum, acc, p->slot_to_row, p->topk_w, p->residual, T, D, K, out, sms,
                       s) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

size_t moe_layer_ex_workspace_size(int T, int D, int E, int K, int f, int f_s, unsigned flags, int int8) {
    if (check_shape(T, D, E, K, f, f_s) != MOE_OK) return 0;
    if (!int8) return moe_workspace_size(T, D, E, K, f, f_s);
    return static_cast<long long>(T) * D >= (1ll << 33) ? 0 : layer_layout(T, D, E, K, f, f_s, flags).total;
}

int moe_layer_forward_ex(const moe_layer_params* p, const moe_route_rule* rule,
                         const moe_int8_weights* weights, moe_bf16* out, void* workspace,
                         size_t ws_bytes, void* stream) {
    if (!p) return MOE_ERR_ARG;
    RouteLogitsLaunch rl{};
    const int rc = rule ? check_layer_rule(p, rule) : MOE_OK;
    if (rc) return rc;
    if (rule) rl = rule_launch(rule);
    if (weights) return layer_int8(p, rule ? &rl : nullptr, weights, out, workspace, ws_bytes,
                                   as_stream(stream));
    return layer_forward(p, rule ? &rl : nullptr, out, workspace, ws_bytes, stream);
}

int moe_layer_plan_ex(const moe_layer_params* p, const moe_route_rule* rule, unsigned* step_mask,
                      int* launches) {
    if (!p) return MOE_ERR_ARG;
    if (!rule) return moe_layer_plan(p, step_mask, launches);
    const int rc = check_layer_rule(p, rule);
    if (rc) return rc;
    const RouteLogitsLaunch rl = rule_launch(rule);
    return layer_plan(p, &rl, step_mask, launches);
}

}  // extern "C"
