"""The 8-bit integer operators against the same arithmetic in 64 bits (int8_ref), whose
allowances count the roundings of the CUDA path."""
import numpy as np
import pytest
import torch

import int8_ref as ref
from workloads import LayerConfig, make_inputs

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- rows to 8 bits


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (5, 2048), (2, 2064), (7, 4096), (2, 8192),
                                       (1, 16400), (1, 40000), (1000, 256)])
def test_quantize_rows(moe, rows, cols):
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))).bfloat16()
    q, s = moe.quantize_rows(x.cuda())
    o_q, o_s = ref.quantise(ref.f64(x))
    np.testing.assert_array_equal(q.cpu().numpy(), o_q)
    top = x.float().abs().amax(1).numpy()
    np.testing.assert_array_equal(s.cpu().numpy(), top / np.float32(127))


def test_quantize_every_bf16_ratio(moe):
    """Rows that hold all mantissas against one maximum, ties among them: exact everywhere."""
    m = torch.arange(128, 256, dtype=torch.float32)
    x = torch.cat([m, -m, m / 2, m / 4, m / 8, m / 64, m / 256, m / 512]).repeat(128, 1)
    top = (m * 2)[:, None]
    x = torch.cat([x, top.expand(-1, 16)], 1)
    x = torch.where(x.abs() > top, torch.zeros_like(x), x).bfloat16()
    q, _ = moe.quantize_rows(x.cuda())
    np.testing.assert_array_equal(q.cpu().numpy(), ref.quantise(ref.f64(x))[0])


def test_quantize_extreme_rows(moe):
    x = torch.zeros(8, 64)
    x[1, :4] = torch.tensor([3e38, -3e38, 1e38, 1e30])
    x[2, :3] = torch.tensor([9.2e-41, -4.6e-41, 9.2e-41])  # subnormal bf16
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5, :2] = torch.tensor([1e-38, -5e-39])
    x[6] = -1.0
    x[7, 63] = 2.0 ** 110
    x = x.bfloat16()
    q, s = moe.quantize_rows(x.cuda())
    o_q, _ = ref.quantise(ref.f64(x))
    np.testing.assert_array_equal(q.cpu().numpy(), o_q)
    s = s.cpu()
    assert torch.isnan(s[3]) and torch.isnan(s[4]) and s[0] == 0
    for r in (1, 2, 5, 6, 7):
        assert s[r].item() == np.float32(x[r].float().abs().max().item()) / np.float32(127)


# ---------------------------------------------------------------- dense products


SHAPES = [(1, 8, 16), (1, 4096, 4096), (3, 520, 1040), (8, 256, 2048), (9, 264, 2064), (77, 4104, 2064),
          (127, 128, 128), (128, 256, 256), (129, 1032, 400), (300, 264, 144), (513, 776, 1024),
          (16, 1032, 8208), (40, 4096, 8192), (130, 264, 4112)]


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_int8_matmul(moe, T, N, K):
    g = torch.Generator().manual_seed(T + N + K)
    xq = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int8)
    wq = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    xs, ws = torch.rand(T, generator=g) + 0.1, torch.rand(N, generator=g) * 1e-3
    y = moe.int8_matmul(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda())
    ref.assert_within(y, *ref.linear(ref.f64(xq), ref.f64(xs), ref.f64(wq), ref.f64(ws)), f"{T} {N} {K}")


def test_int8_matmul_extreme_sums(moe):
    """Every product 2^14, K the longest: the int32 sum is exact."""
    xq = torch.full((2, 65536), -128, dtype=torch.int8)
    wq = torch.full((16, 65536), -128, dtype=torch.int8)
    wq[1::2] = 127
    one = torch.ones(16)
    y = moe.int8_matmul(xq.cuda(), one[:2].cuda(), wq.cuda(), one.cuda()).float().cpu()
    assert (y[:, 0::2] == 2.0 ** 30).all()
    assert (y[:, 1::2] == torch.tensor(-128.0 * 127 * 65536).bfloat16().float()).all()


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_int8_linear(moe, T, N, K):
    g = torch.Generator().manual_seed(T * N + K)
    x = torch.randn(T, K, generator=g).bfloat16()
    wq, ws = ref.channels(N, K, g)
    y = moe.int8_linear(x.cuda(), wq.cuda(), ws.cuda())
    xq, xs = ref.quantise(ref.f64(x))
    want, allow = ref.linear(xq, xs, ref.f64(wq), ref.f64(ws))
    ref.assert_within(y, want, allow + np.abs(want) * ref.F32_HALF, f"{T} {N} {K}")


@pytest.mark.parametrize("T", [0, 1, 5, 40, 200])
def test_linear_is_quantize_then_matmul(moe, T):
    """Bit for bit, into given buffers with rows behind them left as they were; a NaN or inf row
    stays in its row."""
    N, K = 392, 1040
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    if T >= 5:
        x[1, 7], x[3, 1030] = float("nan"), float("inf")
    wq, ws = (t.cuda() for t in ref.channels(N, K, g))
    buf = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = moe.int8_linear(x, wq, ws, out=buf[:T])
    assert (T == 0 or y.data_ptr() == buf.data_ptr()) and bool((buf[T:] == 7).all())
    z = moe.int8_matmul(*moe.quantize_rows(x), wq, ws)
    assert torch.equal(y.view(torch.int16), z.view(torch.int16)) or torch.equal(
        torch.nan_to_num(y), torch.nan_to_num(z))
    if T >= 5:
        nan = torch.isnan(y)
        assert nan[1].all() and nan[3].all() and int(nan.sum()) == 2 * N


# ---------------------------------------------------------------- experts


class Case:
    def __init__(self, T, D, E, K, f, seed=0, skew=None):
        g = torch.Generator().manual_seed(seed + T + D + E + f)
        self.T, self.D, self.E, self.K, self.f = T, D, E, K, f
        self.x = torch.randn(T, D, generator=g).bfloat16()
        gu, gus, dn, dns = [], [], [], []
        for _ in range(E):
            a, b = ref.channels(2 * f, D, g)
            c, d = ref.channels(D, f, g)
            gu.append(a), gus.append(b), dn.append(c), dns.append(d)
        self.weights = [torch.stack(v) for v in (gu, gus, dn, dns)]
        score = torch.rand(T, E, generator=g)
        if skew == "one":
            score[:, 1] += 2
        if skew == "few":
            score[:, :K] += 2
        self.idx = torch.argsort(-score, dim=1)[:, :K].int().contiguous()
        self.w = torch.rand(T, K, generator=g) + 0.05
        self.residual = torch.randn(T, D, generator=g).bfloat16()

    def want(self, keep=None, residual=False):
        xq, xs = ref.quantise(ref.f64(self.x))
        return ref.experts(xq, xs, self.idx.numpy(), ref.f64(self.w), *map(ref.f64, self.weights),
                           keep=keep, residual=ref.f64(self.residual) if residual else None)

    def on_gpu(self, moe, capacity=None):
        idx, w = self.idx.cuda(), self.w.cuda()
        counts = torch.bincount(idx.reshape(-1), minlength=self.E).int()
        perm = moe.permute(idx, w, counts, self.E, capacity=capacity)
        xq, xs = moe.quantize_rows(self.x.cuda())
        return (xq, xs, w, perm, *(t.cuda() for t in self.weights))


CASES = [(1, 2048, 8, 4, 128, None),     # K cut into slices
         (1, 128, 1, 1, 128, None),
         (5, 384, 6, 3, 256, None),      # half a tile of output columns
         (64, 256, 16, 4, 128, "few"),
         (200, 256, 4, 2, 384, "one"),   # a hot expert, idle ones
         (2, 256, 8, 2, 1152, None),     # a handful of rows, by chunks of a weight row
         (3, 1024, 8, 4, 512, "few"),
         (1, 384, 4, 3, 640, None),
         (64, 256, 64, 4, 128, "few"),   # few rows on average, hot experts
         (24, 2048, 2, 2, 128, None),    # one-CTA tiles cut into slices
         (300, 640, 4, 2, 128, None),    # CTA pairs
         (700, 256, 3, 2, 256, "one")]


@pytest.mark.parametrize("T,D,E,K,f,skew", CASES)
@pytest.mark.parametrize("deterministic", [False, True])
def test_experts(moe, T, D, E, K, f, skew, deterministic):
    c = Case(T, D, E, K, f, skew=skew)
    y = moe.experts_int8(*c.on_gpu(moe), deterministic=deterministic)
    ref.assert_within(y, *c.want(), f"{T} {D} {E} {K} {f}")
    y = moe.experts_int8(*c.on_gpu(moe), deterministic=deterministic, residual=c.residual.cuda())
    ref.assert_within(y, *c.want(residual=True), "with residual")


def test_no_tokens(moe):
    c = Case(0, 256, 4, 2, 128)
    perm = dict(offsets=torch.zeros(5, dtype=torch.int32, device="cuda"),
                **{k: torch.empty(0, dtype=torch.int32, device="cuda")
                   for k in ("sorted_token", "slot_to_row")},
                sorted_w=torch.empty(0, device="cuda"))
    xq, xs = moe.quantize_rows(c.x.cuda())
    y = moe.experts_int8(xq, xs, c.w.cuda(), perm, *(t.cuda() for t in c.weights))
    assert y.shape == (0, 256)


@pytest.mark.parametrize("T,E,C", [(4, 8, 1), (40, 8, 5), (600, 4, 150), (600, 4, 0)])
@pytest.mark.parametrize("deterministic", [False, True])
def test_dropped_rows_add_nothing(moe, oracle_mod, T, E, C, deterministic):
    """An expert capacity leaves rows behind the last group; NaN weights there must not show."""
    c = Case(T, 256, E, 2, 128, skew="one")
    args = list(c.on_gpu(moe, capacity=C))
    n = int(args[3]["offsets"][-1])
    args[3]["sorted_w"][n:] = float("nan")
    keep = oracle_mod.capacity_keep(c.idx.numpy(), E, C)
    assert not keep.all()
    y = moe.experts_int8(*args, deterministic=deterministic, residual=c.residual.cuda())
    ref.assert_within(y, *c.want(keep=np.asarray(keep, bool), residual=True))


def test_a_bad_token_stays_alone(moe):
    c = Case(33, 256, 4, 2, 128)
    c.x[4, 9], c.x[20, 100] = float("nan"), float("-inf")
    y = moe.experts_int8(*c.on_gpu(moe))
    nan = torch.isnan(y).cpu()
    assert nan[4].all() and nan[20].all() and int(nan.sum()) == 2 * 256
    want, allow = c.want()
    rows = [t for t in range(33) if t not in (4, 20)]
    ref.assert_within(ref.f64(y)[rows], want[rows], allow[rows])


def test_zero_tokens_and_zero_weights(moe):
    c = Case(20, 256, 4, 2, 128)
    c.x[3] = 0
    c.w[5] = 0
    y = moe.experts_int8(*c.on_gpu(moe))
    assert (y[3] == 0).all() and (y[5] == 0).all()
    ref.assert_within(y, *c.want())


def test_deterministic_repeats(moe):
    c = Case(300, 256, 4, 2, 128)
    a = c.on_gpu(moe)
    ys = [moe.experts_int8(*a, deterministic=True) for _ in range(4)]
    assert all(torch.equal(y, ys[0]) for y in ys)


def test_two_streams_at_once(moe):
    """Calls with workspaces of their own on two streams, as many as fit in flight."""
    cs = [Case(1, 2048, 8, 4, 128), Case(64, 256, 16, 4, 128), Case(300, 640, 4, 2, 128)]
    args = [c.on_gpu(moe) for c in cs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for rep in range(10):
        for i, a in enumerate(args):
            got.append((i, moe.experts_int8(*a, stream=streams[(rep + i) % 2])))
    torch.cuda.synchronize()
    wants = [c.want() for c in cs]
    for i, y in got:
        ref.assert_within(y, *wants[i], f"case {i}")


def test_graph_replay(moe):
    c = Case(40, 256, 8, 2, 128)
    args = c.on_gpu(moe)
    x = c.x.cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xq, xs = moe.quantize_rows(x)
        y = moe.experts_int8(xq, xs, *args[2:])
        z = moe.int8_linear(x, args[4][0], args[5][0])
    other = Case(40, 256, 8, 2, 128, seed=9)
    c.x = other.x
    x.copy_(other.x)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    ref.assert_within(y, *c.want())
    xq, xs = ref.quantise(ref.f64(other.x))
    want, allow = ref.linear(xq, xs, ref.f64(c.weights[0][0]), ref.f64(c.weights[1][0]))
    ref.assert_within(z, want, allow + np.abs(want) * ref.F32_HALF)


# ---------------------------------------------------------------- the layer


@pytest.mark.parametrize("T,E,shared,options", [
    (37, 16, False, {}),
    (1, 16, True, {}),
    (300, 128, True, {}),                      # logits from the tensor cores
    (520, 4, True, {}),                        # CTA pairs
    (64, 16, True, {"deterministic": True}),
    (64, 16, False, {"deterministic": True}),
    (100, 16, True, {"capacity_factor": 0.5}),
    (64, 16, False, {"score": "sigmoid"}),
])
@pytest.mark.parametrize("grouped", [False, True])
def test_layer(moe, oracle_mod, T, E, shared, options, grouped):
    """Route, quantise, permute, experts, shared expert, residual through Int8MoELayer, for the
    routing that it reports (checked against the oracle where the rule is the plain one)."""
    K, D, f = 2, 256, 128
    if grouped and options.get("score"):
        pytest.skip("a rule carries its own scores")
    cfg = LayerConfig("int8", T=T, D=D, E=E, K=K, f=f, f_s=256 if shared else 0, seed=T)
    inp = make_inputs(cfg).to("cuda")
    rule = moe.route_rule(E, K, score="sigmoid", n_group=2, topk_group=1, scale=1.5) if grouped else None
    layer = moe.Int8MoELayer.from_inputs(inp, rule=rule, **options)
    idx = torch.empty((T, K), dtype=torch.int32, device="cuda")
    w = torch.empty((T, K), device="cuda")
    h = torch.randn(T, D, device="cuda").bfloat16()
    for _ in range(2):
        y = layer(inp.x, topk_idx=idx, topk_w=w, residual=h)
    assert layer.device_status() == 0
    i = idx.cpu().numpy()
    if grouped:
        assert (i // (E // 2) == i[:, :1] // (E // 2)).all()
    else:
        from parity import check_route
        orc = oracle_mod.route(inp.x, inp.w_router, K, None, inp.w_shared_gate,
                               options.get("score", "softmax"))
        check_route(orc, i, w.cpu().numpy())
    keep = None
    if "capacity_factor" in options:
        C = moe.expert_capacity(T, K, E, options["capacity_factor"])
        keep = np.asarray(oracle_mod.capacity_keep(i, E, C), bool)
    weights = []
    for t in (inp.w_gate_up, inp.w_down):
        q, s = ref.quantise(ref.f64(t))
        weights += [q, s]
    sh = None
    if shared:
        gate = 1 / (1 + np.exp(-ref.f64(inp.x) @ ref.f64(inp.w_shared_gate)))
        sh = [gate]
        for t in (inp.w_shared_gate_up, inp.w_shared_down):
            sh += list(ref.quantise(ref.f64(t)))
    xq, xs = ref.quantise(ref.f64(inp.x))
    want, allow = ref.experts(xq, xs, i, ref.f64(w), weights[0], weights[1], weights[2], weights[3],
                              keep=keep, residual=ref.f64(h), shared=sh)
    # the scales are fp32 roundings of the 64-bit ones: two more factors per product
    ref.assert_within(y, want, allow + np.abs(want) * 8 * ref.F32_HALF + 1e-6 * np.abs(want - ref.f64(h)))


def test_bf16_layer_with_a_rule(moe):
    """MoELayer with groups: the plain layer on the tokens' own routing, weight by weight."""
    cfg = LayerConfig("rule_layer", T=70, D=256, E=16, K=4, f=128, f_s=128, seed=2)
    inp = make_inputs(cfg).to("cuda")
    bias = 0.05 * torch.randn(16, device="cuda")
    rule = moe.route_rule(16, 4, "sigmoid", bias, 4, 2, scale=2.0)
    layer = moe.MoELayer.from_inputs(inp, rule=rule)
    idx = torch.empty((70, 4), dtype=torch.int32, device="cuda")
    w = torch.empty((70, 4), device="cuda")
    y = layer(inp.x, topk_idx=idx, topk_w=w)
    i2, w2, counts, sg = moe.route(inp.x, inp.w_router, 4, None, inp.w_shared_gate, rule=rule)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    x = inp.x.double()
    want = torch.zeros(70, 256, dtype=torch.float64, device="cuda")
    def expert(gu, dn, v):
        a = v @ gu.double().t()
        n = a.shape[1] // 2
        return (torch.nn.functional.silu(a[:, :n]) * a[:, n:]) @ dn.double().t()
    for e in range(16):
        t, k = (idx == e).nonzero(as_tuple=True)
        want.index_add_(0, t, expert(inp.w_gate_up[e], inp.w_down[e], x[t]) * w[t, k].double()[:, None])
    gate = torch.sigmoid(x @ inp.w_shared_gate.double())
    want += gate[:, None] * expert(inp.w_shared_gate_up, inp.w_shared_down, x)
    from parity import output_error
    err, rms, used = output_error(ref.f64(y), want.cpu().numpy())
    assert used <= 1, (err, rms)


# ---------------------------------------------------------------- refusals of the binding


def test_binding_refusals(moe):
    """Shapes, types, strides and devices that do not fit raise before anything is launched."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    w, ws = torch.zeros(8, 64, dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    r = torch.zeros(4, 64, device="cuda")
    for call in (lambda: moe.int8_linear(x, w[:, :32].contiguous(), ws), lambda: moe.int8_linear(x, w, s),
                 lambda: moe.int8_linear(x[0], w, ws), lambda: moe.int8_matmul(q, ws, w, ws),
                 lambda: moe.int8_matmul(q, s, w, s), lambda: moe.int8_linear(x, w[:6], ws[:6]),
                 lambda: moe.int8_linear(x, w, ws, out=torch.empty(4, 9, device="cuda").bfloat16()),
                 lambda: moe.int8_linear(x[:, :40].contiguous(), w[:, :40].contiguous(), ws),
                 lambda: moe.quantize_rows(x[:, :40].contiguous()), lambda: moe.route_logits(r, 17),
                 lambda: moe.route_logits(r, 4, n_group=7), lambda: moe.route_logits(r[0], 4),
                 lambda: moe.route_logits(r, 9, n_group=8, topk_group=1),
                 lambda: moe.route_logits(r, 4, select_bias=s),
                 lambda: moe.route_logits(r, 4, scale=float("nan"))):
        with pytest.raises(moe.MoEError):
            call()
    for call in (lambda: moe.int8_linear(x.float(), w, ws), lambda: moe.int8_linear(x, w.float(), ws),
                 lambda: moe.quantize_rows(x.half()), lambda: moe.route_logits(r.half(), 4),
                 lambda: moe.int8_matmul(q, s.double(), w, ws)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: moe.int8_linear(x.t().contiguous().t(), w, ws), lambda: moe.int8_linear(x, w.cpu(), ws),
                 lambda: moe.quantize_rows(x[:, :32]), lambda: moe.route_logits(r[:, ::2], 4),
                 lambda: moe.int8_matmul(q, s.cpu(), w, ws)):
        with pytest.raises(ValueError):
            call()
    c = Case(6, 256, 4, 2, 128)
    a = list(c.on_gpu(moe))
    for i, bad in ((0, a[0][:5].contiguous()), (1, a[1][:5].contiguous()), (2, a[2][:5].contiguous()),
                   (4, a[4][:3].contiguous()), (5, a[5][:3].contiguous()), (7, a[7][:3].contiguous())):
        b = list(a)
        b[i] = bad
        with pytest.raises(moe.MoEError):
            moe.experts_int8(*b)
    with pytest.raises(moe.MoEError):
        moe.experts_int8(*a, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
