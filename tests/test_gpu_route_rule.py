"""Routing by a rule (expert groups, masks, unnormalised and scaled weights) against the
definition in 64 bits: the experts have to be equal, ties and near ties included."""
import numpy as np
import pytest
import torch

import int8_ref as ref
from parity import W_TOL, check_route
from workloads import LayerConfig, make_inputs

pytestmark = pytest.mark.gpu


def check(moe, logits, K, bias=None, **rule):
    idx, w, counts = moe.route_logits(logits.cuda(), K,
                                      select_bias=None if bias is None else bias.cuda(), **rule)
    o_idx, o_w, tol = ref.route(logits, K, bias=bias, score=rule.get("score", "softmax"),
                                n_group=rule.get("n_group", 1), topk_group=rule.get("topk_group", 1),
                                group_top=rule.get("group_top") or (1 if bias is None else 2),
                                renorm=rule.get("renorm", True), scale=rule.get("scale", 1.0))
    np.testing.assert_array_equal(idx.cpu().numpy(), o_idx)
    ref.assert_within(w, o_w, tol, "weights")
    np.testing.assert_array_equal(counts.cpu().numpy(),
                                  np.bincount(o_idx.reshape(-1), minlength=logits.shape[1]))
    return idx, w


def draw(T, E, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (1.5 * torch.randn(T, E, generator=g)).to(dtype), 0.1 * torch.randn(E, generator=g)


@pytest.mark.parametrize("T", [0, 1, 7, 33, 300])
@pytest.mark.parametrize("E,K,G,M", [(256, 8, 8, 4), (1, 1, 1, 1), (60, 6, 4, 2), (96, 16, 3, 1),
                                     (512, 10, 16, 5), (512, 16, 32, 32), (64, 4, 32, 3), (33, 3, 11, 2)])
@pytest.mark.parametrize("score,with_bias,group_top", [("sigmoid", True, 2), ("softmax", False, 1),
                                                       ("softmax", True, 2), ("softmax", False, 2),
                                                       ("sigmoid", False, 2)])
def test_route_logits(moe, T, E, K, G, M, score, with_bias, group_top):
    logits, bias = draw(T, E, 3 * T + E)
    check(moe, logits, K, bias if with_bias else None, score=score, n_group=G, topk_group=M,
          group_top=group_top, renorm=T % 2 == 0, scale=2.5)


@pytest.mark.parametrize("score,with_bias,group_top", [("sigmoid", True, 2), ("softmax", False, 1),
                                                       ("softmax", False, 2)])
def test_bf16_logits_with_many_ties(moe, score, with_bias, group_top):
    logits, bias = draw(500, 128, 5, torch.bfloat16)
    bias = torch.round(bias * 8) / 8
    check(moe, logits, 8, bias if with_bias else None, score=score, n_group=8, topk_group=3,
          group_top=group_top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,M", [(1, 1), (8, 3)])
def test_keys_that_fp32_cannot_tell_apart(moe, score, G, M):
    """One bias per expert that brings the keys of token 0 within a few fp32 steps of each
    other: the order is in the digits that fp32 drops.  (Other tokens are ordinary.)"""
    T, E = 64, 256
    logits, _ = draw(1, E, 11)
    s = torch.sigmoid(logits.double()) if score == "sigmoid" else torch.softmax(logits.double(), 1)
    bias = (1.0 - s[0]).float()
    logits = logits + torch.cat([torch.zeros(1, 1), torch.randn(T - 1, 1)]) * (score == "sigmoid")
    check(moe, logits, 8, bias, score=score, n_group=G, topk_group=M)


def test_equal_logits_take_the_lowest_experts(moe):
    idx, w = check(moe, torch.zeros(40, 64), 4, n_group=8, topk_group=2)
    assert idx.cpu().tolist() == [[0, 1, 2, 3]] * 40


def test_masked_experts(moe):
    """-inf and NaN logits: out; rows with fewer than K experts left, and with none."""
    logits, bias = draw(12, 64, 21)
    inf = float("inf")
    logits[0] = -inf                      # nothing left: the lowest experts, weight 0
    logits[1] = float("nan")
    logits[2, 3:] = -inf                  # three left, K = 6
    logits[3, ::2] = -inf
    logits[4, 16:] = float("nan")         # whole groups out
    logits[5, 40] = inf
    logits[6, 1] = logits[6, 50] = inf
    logits[7] = torch.finfo(torch.float32).min
    for b in (None, bias):
        for score in ("softmax", "sigmoid"):
            for G, M in ((1, 1), (4, 2)):
                for renorm in (True, False):
                    idx, w = check(moe, logits, 6, b, score=score, n_group=G, topk_group=M,
                                   renorm=renorm)
                    assert not torch.isnan(w).any()
                    assert (w[0] == 0).all() and (w[1] == 0).all()
                    assert ((w[2] > 0).sum() <= 3)


def test_disabled_experts_by_bias(moe):
    logits, bias = draw(50, 64, 22)
    bias[5], bias[9], bias[20] = -float("inf"), float("nan"), float("inf")
    idx, _ = check(moe, logits, 8, bias, score="sigmoid", n_group=4, topk_group=3)
    assert not ((idx == 5) | (idx == 9)).any() and (idx[:, 0] == 20).all()


@pytest.mark.parametrize("G,M", [(1, 1), (4, 2), (2, 1)])
def test_more_forced_experts_than_slots(moe, G, M):
    """A bias of +inf for more experts than K: the lowest of them, whatever their scores."""
    logits, bias = draw(40, 64, 23)
    bias[10:30] = float("inf")
    idx, w = check(moe, logits, 6, bias, score="sigmoid", n_group=G, topk_group=M)
    assert torch.isfinite(w).all() and bool((bias[idx.cpu().long()] == float("inf")).all())


def test_far_logits_keep_their_ratios(moe):
    """Sigmoid scores that underflow in fp32 still renormalise to the ratios e^(r_i - r_j)."""
    logits = torch.full((3, 32), -300.0)
    logits[:, 3], logits[:, 7] = -200.0, -201.0
    _, w = check(moe, logits, 2, score="sigmoid")
    assert abs(w[0, 0].item() - 1 / (1 + np.exp(-1))) < 1e-6


def test_many_tokens_and_large_offsets(moe):
    """More tokens than a launch has warps; the last row's offset is checked on its own."""
    T, E = 40000, 64
    logits, bias = draw(T, E, 31)
    idx, w, counts = moe.route_logits(logits.cuda(), 6, score="sigmoid", select_bias=bias.cuda(),
                                      n_group=8, topk_group=4)
    assert int(counts.sum()) == T * 6
    rows = list(range(0, T, 997)) + [T - 1]
    o_idx, o_w, tol = ref.route(logits[rows], 6, "sigmoid", bias, 8, 4, 2)
    np.testing.assert_array_equal(idx[rows].cpu().numpy(), o_idx)
    ref.assert_within(w[rows], o_w, tol)
    np.testing.assert_array_equal(counts.cpu().numpy(),
                                  np.bincount(idx.cpu().numpy().reshape(-1), minlength=E))


def test_graph_replay_and_other_stream(moe):
    logits, bias = draw(200, 128, 41)
    dev, b = logits.cuda(), bias.cuda()
    want = moe.route_logits(dev, 8, score="sigmoid", select_bias=b, n_group=8, topk_group=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = moe.route_logits(dev, 8, score="sigmoid", select_bias=b, n_group=8, topk_group=4, stream=s)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = moe.route_logits(dev, 8, score="sigmoid", select_bias=b, n_group=8, topk_group=4)
    other, _ = draw(200, 128, 42)
    want = moe.route_logits(other.cuda(), 8, score="sigmoid", select_bias=b, n_group=8, topk_group=4)
    dev.copy_(other)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T,E", [(37, 64), (300, 128)])  # CUDA-core and tensor-core logits
@pytest.mark.parametrize("shared", [False, True])
def test_route_with_a_rule(moe, oracle_mod, T, E, shared):
    """The router's own logits: one group and no bias is the plain router; with groups the
    experts are a valid selection by the oracle's scores up to near ties."""
    cfg = LayerConfig("rule", T=T, D=256, E=E, K=4, f=128, f_s=128 if shared else 0, seed=5)
    inp = make_inputs(cfg).to("cuda")
    orc = oracle_mod.route(inp.x, inp.w_router, 4, None, inp.w_shared_gate)
    idx, w, counts, sg = moe.route(inp.x, inp.w_router, 4, None, inp.w_shared_gate,
                                   rule=moe.route_rule(E, 4))
    check_route(orc, idx.cpu().numpy(), w.cpu().numpy(), counts.cpu().numpy())
    if shared:
        assert np.abs(sg.cpu().numpy() - orc["shared_gate"]).max() <= 1e-5
    rule = moe.route_rule(E, 4, n_group=8, topk_group=2, scale=2.0)
    idx, w, counts, _ = moe.route(inp.x, inp.w_router, 4, None, inp.w_shared_gate, rule=rule)
    logits = torch.tensor(np.log(orc["probs"]))
    o_idx, o_w, _ = ref.route(logits, 4, n_group=8, topk_group=2, scale=2.0)
    same = (idx.cpu().numpy() == o_idx).all(1)
    assert same.mean() > 0.97  # the others: near ties of fp32 logits
    assert np.abs(w.cpu().numpy() - o_w)[same].max() <= 2 * W_TOL
    np.testing.assert_array_equal(counts.cpu().numpy(),
                                  np.bincount(idx.cpu().numpy().reshape(-1), minlength=E))
