"""Cases for timing the routing and 8-bit integer operators of the MoE layer.

``run`` computes a case either in plain torch (``own`` false) or through this package's
entry points (``own`` true).  Three operators:

* ``route``: experts of each token from given router logits -- softmax or sigmoid scores, a
  selection-only bias, expert groups, top-k, (re)normalised and scaled weights.
* ``linear``: a linear layer in 8-bit integers, tokens quantised per row on the fly, weights
  per output channel.
* ``experts``: the routed SwiGLU experts of one layer in the same arithmetic, for a routing
  that the program already has.
"""
import math

import torch

own = False

LARGEST_LINEAR = 8192 * 8192 * 4096
LARGEST_EXPERTS = 65536 * 4096 * 1024
LARGEST_WEIGHTS = 64 * 4096 * 1024


# ------------------------------------------------------------------ cases


def _route(name, T, E, K, score, dtype, bias, n_group=1, topk_group=1, group_top=1, renorm=True,
           scale=1.0):
    return dict(name=name, op="route", T=T, E=E, K=K, score=score, dtype=dtype, bias=bias,
                n_group=n_group, topk_group=topk_group, group_top=group_top, renorm=renorm,
                scale=scale)


def listed():
    return [
        # one token of a stream: latency; sigmoid scores with a balance bias in 8 groups
        _route("route_single", 1, 256, 8, "sigmoid", "float32", True, 8, 4, 2, True, 2.5),
        # a decode batch with logits in the model's type, scores left as they are
        _route("route_decode", 64, 128, 8, "softmax", "bfloat16", False, renorm=False),
        # the fine-grained layer's tokens in 16 groups
        _route("route_finegrained", 4096, 512, 10, "sigmoid", "float32", True, 16, 5, 2),
        # a ragged long prompt batch, groups judged by their best expert
        _route("route_prefill", 16381, 256, 8, "softmax", "float32", False, 8, 3, 1, False, 16.0),
        # single token through a square projection: the weights' bytes and latency
        dict(name="linear_single", op="linear", T=1, N=4096, K=4096),
        # a ragged batch and sizes that no tile divides
        dict(name="linear_ragged", op="linear", T=77, N=4104, K=2064),
        # a prompt batch: arithmetic
        dict(name="linear_prefill", op="linear", T=8192, N=8192, K=4096),
        # one token's eight experts
        dict(name="experts_single", op="experts", T=1, D=4096, E=128, K=8, f=1024, skew=0.0),
        # the decode layer: two rows per expert
        dict(name="experts_decode", op="experts", T=64, D=2048, E=256, K=8, f=512, skew=0.0),
        # an odd batch with a few hot experts and many idle ones
        dict(name="experts_skewed", op="experts", T=1021, D=2048, E=128, K=8, f=512, skew=2.4),
        # the fine-grained layer: 80 rows per expert, 6.4 GB of weights
        dict(name="experts_finegrained", op="experts", T=4096, D=4096, E=512, K=10, f=1024,
             skew=0.0),
        # a prompt batch: a thousand rows per expert
        dict(name="experts_prefill", op="experts", T=8192, D=4096, E=64, K=8, f=1024, skew=0.0),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "linear", "experts"])
    if op == "route":
        E = rng.choice([16, 60, 64, 96, 128, 160, 256, 384, 512])
        n_group = rng.choice([g for g in (1, 2, 4, 8, 16) if E % g == 0 and E // g >= 2])
        topk_group = rng.randint(1, n_group)
        K = rng.randint(1, min(16, topk_group * (E // n_group)))
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, K=K,
                    score=rng.choice(["softmax", "sigmoid"]),
                    dtype=rng.choice(["float32", "bfloat16"]), bias=rng.random() < 0.5,
                    n_group=n_group, topk_group=topk_group, group_top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    if op == "linear":
        while True:
            c = dict(op=op, T=_log_int(rng, 1, 8192), N=_log_int(rng, 128, 8192, 8),
                     K=_log_int(rng, 128, 8192, 16))
            if c["T"] * c["N"] * c["K"] <= LARGEST_LINEAR:
                return c
    while True:
        E = _log_int(rng, 8, 256)
        c = dict(op=op, T=_log_int(rng, 1, 4096), D=_log_int(rng, 256, 4096, 128), E=E,
                 K=rng.randint(1, min(10, E)), f=_log_int(rng, 128, 1024, 128),
                 skew=rng.choice([0.0, 0.0, 2.4]))
        if (c["T"] * c["K"] * c["D"] * c["f"] <= LARGEST_EXPERTS
                and c["E"] * c["D"] * c["f"] <= LARGEST_WEIGHTS
                and not (c["skew"] and c["T"] * c["E"] * c["D"] > 2 ** 29)):
            return c


# ------------------------------------------------------------------ inputs


def _expert_bias(E, skew, gen):
    """Logit offsets that make expert popularity fall as rank ** -skew."""
    rank = torch.empty(E, device="cuda")
    rank[torch.randperm(E, generator=gen, device="cuda")] = torch.arange(1, E + 1, device="cuda").float()
    return -skew * torch.log(rank)


def _activations(T, D, gen):
    """Unit normal activations with the few large channels that hidden states have."""
    x = torch.randn(T, D, generator=gen, device="cuda")
    big = torch.randint(0, D, (max(1, D // 512),), generator=gen, device="cuda")
    x[:, big] *= 6.0
    return x.bfloat16()


def _channels(rows, cols, gen):
    """An 8-bit weight matrix [rows, cols] and its channel scales [rows]."""
    w = torch.randn(rows, cols, generator=gen, device="cuda") / math.sqrt(cols)
    s = w.abs().amax(1) / 127
    return torch.round(w / s[:, None]).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = case
    if c["op"] == "route":
        logits = torch.randn(c["T"], c["E"], generator=gen, device="cuda")
        logits += 0.3 * torch.randn(c["E"], generator=gen, device="cuda")
        bias = 0.05 * torch.randn(c["E"], generator=gen, device="cuda") if c["bias"] else None
        return dict(c, logits=logits.to(getattr(torch, c["dtype"])), bias_t=bias)
    if c["op"] == "linear":
        x = _activations(c["T"], c["K"], gen)
        wq, ws = _channels(c["N"], c["K"], gen)
        return dict(c, x=x, wq=wq, ws=ws)
    T, D, E, K, f = c["T"], c["D"], c["E"], c["K"], c["f"]
    x = _activations(T, D, gen)
    gu = torch.empty(E, 2 * f, D, dtype=torch.int8, device="cuda")
    gus = torch.empty(E, 2 * f, device="cuda")
    dn = torch.empty(E, D, f, dtype=torch.int8, device="cuda")
    dns = torch.empty(E, D, device="cuda")
    for e in range(E):
        gu[e], gus[e] = _channels(2 * f, D, gen)
        dn[e], dns[e] = _channels(D, f, gen)
    r = torch.randn(T, E, generator=gen, device="cuda") + _expert_bias(E, c["skew"], gen)
    r, idx = torch.sort(r, dim=1, descending=True, stable=True)
    w = torch.softmax(r[:, :K], 1)
    idx = idx[:, :K]
    # the permutation by expert that the program keeps beside its routing
    order = torch.sort(idx.reshape(-1), stable=True).indices
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    slot_to_row = torch.empty(T * K, dtype=torch.int32, device="cuda")
    slot_to_row[order] = torch.arange(T * K, dtype=torch.int32, device="cuda")
    perm = dict(offsets=offsets, sorted_token=(order // K).int(),
                sorted_w=w.reshape(-1)[order].contiguous(), slot_to_row=slot_to_row)
    return dict(c, x=x, gu=gu, gus=gus, dn=dn, dns=dns, topk_w=w.contiguous(), perm=perm,
                longest=int(counts.max()))


# ------------------------------------------------------------------ one pass


def _route_plain(s):
    T, E, K, G = s["T"], s["E"], s["K"], s["n_group"]
    r = s["logits"].double()  # 64 bits: the scores next to the borders decide the experts
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-r))
    else:
        p = torch.exp(r - r.amax(1, keepdim=True))
        score = p / p.sum(1, keepdim=True)
    key = score if s["bias_t"] is None else score + s["bias_t"].double()
    best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
    best = best[:, :, :s["group_top"]].sum(2)
    kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["topk_group"]]
    allowed = torch.zeros(T, G, dtype=torch.bool, device=r.device).scatter_(1, kept, True)
    key = torch.where(allowed[:, :, None], key.view(T, G, E // G), -torch.inf).view(T, E)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    w = torch.gather(score, 1, idx)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    return dict(idx=idx.int(), w=(w * s["scale"]).float(), counts=counts.int())


def _quantised(x):
    """Whole numbers in [-127, 127] (as fp32) and the scale of each row."""
    x = x.float()
    top = x.abs().amax(-1, keepdim=True)
    return torch.round(127 * x / torch.where(top == 0, 1, top)), top / 127


def _linear_plain(s):
    q, xs = _quantised(s["x"])
    return (q @ s["wq"].float().t() * xs * s["ws"]).bfloat16()


def _experts_plain(s):
    T, D, E, K, perm = s["T"], s["D"], s["E"], s["K"], s["perm"]
    q, xs = _quantised(s["x"])
    # the rows of each expert, padded to the longest
    off = perm["offsets"].long()
    row = off[:-1, None] + torch.arange(s["longest"], device=q.device)
    real = row < off[1:, None]
    row = torch.where(real, row, 0)
    tok = perm["sorted_token"].long()[row]
    y = torch.bmm(q[tok], s["gu"].float().transpose(1, 2))
    y = y * xs[tok] * s["gus"][:, None, :]
    g, u = y.chunk(2, 2)
    h, hs = _quantised(g / (1 + torch.exp(-g)) * u)
    v = torch.bmm(h, s["dn"].float().transpose(1, 2))
    v = v * (hs * perm["sorted_w"][row][:, :, None]) * s["dns"][:, None, :]
    y = torch.zeros(T, D, device=q.device).index_add_(0, tok[real], v[real])
    return y.bfloat16()


def run(state):
    s = state
    if own:
        import top_routing_grouped_03_b200 as moe
        if s["op"] == "route":
            idx, w, counts = moe.route_logits(
                s["logits"], s["K"], score=s["score"], select_bias=s["bias_t"],
                n_group=s["n_group"], topk_group=s["topk_group"], group_top=s["group_top"],
                renorm=s["renorm"], scale=s["scale"])
            return dict(idx=idx, w=w, counts=counts)
        if s["op"] == "linear":
            return moe.int8_linear(s["x"], s["wq"], s["ws"])
        xq, xs = moe.quantize_rows(s["x"])
        return moe.experts_int8(xq, xs, s["topk_w"], s["perm"], s["gu"], s["gus"], s["dn"], s["dns"])
    return {"route": _route_plain, "linear": _linear_plain, "experts": _experts_plain}[s["op"]](s)


# ------------------------------------------------------------------ what a pass cannot do without


def _experts_hit(c):
    share = [(e + 1.0) ** -c["skew"] for e in range(c["E"])]
    total = sum(share)
    return sum(1 - (1 - min(1.0, c["K"] * p / total)) ** c["T"] for p in share)


def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "float32" else 2
        return {"bytes": c["T"] * (c["E"] * size + c["K"] * 8) + c["E"] * (8 if c["bias"] else 4),
                "flops": 8 * c["T"] * c["E"]}
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": 2 * T * K + N * K + 4 * N + 2 * T * N, "flops": 2 * T * N * K}
    T, D, K, f = c["T"], c["D"], c["K"], c["f"]
    weights = _experts_hit(c) * (3 * D * f + 4 * (2 * f + D))
    return {"bytes": int(4 * T * D + 12 * T * K + weights), "flops": 6 * T * K * D * f}


# ------------------------------------------------------------------ in 64 bits


def _exact_rows(x):
    """The rows' whole numbers and scales, in 64 bits."""
    top = x.abs().max(1).values
    scale = top / 127
    return torch.round(x * 127 / top.clamp(min=1e-300)[:, None]), scale


def _exact_route(c, s):
    import numpy as np
    r = s["logits"].double().cpu().numpy()
    if c["score"] == "sigmoid":
        score = np.where(r < 0, np.exp(-np.logaddexp(0, -r)), 1 / (1 + np.exp(-np.abs(r))))
    else:
        score = np.exp(r - np.logaddexp.reduce(r, axis=1)[:, None])
    key = score + (0 if s["bias_t"] is None else s["bias_t"].double().cpu().numpy())
    T, E, G = c["T"], c["E"], c["n_group"]
    group = np.partition(key.reshape(T, G, E // G), E // G - c["group_top"], axis=2)
    group = group[:, :, E // G - c["group_top"]:].sum(2)
    place = np.argsort(np.argsort(-group, axis=1, kind="stable"), axis=1, kind="stable")
    key = np.where(np.repeat(place < c["topk_group"], E // G, axis=1), key, -np.inf)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :c["K"]]
    w = np.take_along_axis(score, idx, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return dict(idx=idx.astype(np.int32), w=w * c["scale"],
                counts=np.bincount(idx.ravel(), minlength=E).astype(np.int32))


def _exact_experts(c, s):
    q, xs = _exact_rows(s["x"].double())
    y = torch.zeros(c["T"], c["D"], dtype=torch.float64, device=q.device)
    off = s["perm"]["offsets"].tolist()
    for e in range(c["E"]):
        if off[e] == off[e + 1]:
            continue
        tok = s["perm"]["sorted_token"][off[e]:off[e + 1]].long()
        w = s["perm"]["sorted_w"][off[e]:off[e + 1]].double()
        a = (q[tok] @ s["gu"][e].double().t()) * xs[tok][:, None] * s["gus"][e].double()
        h, hs = _exact_rows(a[:, :c["f"]] * torch.sigmoid(a[:, :c["f"]]) * a[:, c["f"]:])
        y.index_add_(0, tok, (h @ s["dn"][e].double().t()) * s["dns"][e].double() * (hs * w)[:, None])
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "linear":
        q, xs = _exact_rows(s["x"].double())
        return (q @ s["wq"].double().t()) * xs[:, None] * s["ws"].double()
    return _exact_experts(case, s)
