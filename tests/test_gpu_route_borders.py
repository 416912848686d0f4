"""Borders between expert groups whose scores fp32 cannot tell apart although they look far apart in
it: the experts have to be those of the definition in 64 bits."""
import numpy as np
import pytest
import torch

import int8_ref as ref

pytestmark = pytest.mark.gpu


def check(moe, logits, K, bias, **rule):
    idx, w, counts = moe.route_logits(logits.cuda(), K, select_bias=None if bias is None else bias.cuda(),
                                      group_top=2, **rule)
    o_idx, o_w, tol = ref.route(logits, K, bias=bias, group_top=2, **rule)
    np.testing.assert_array_equal(idx.cpu().numpy(), o_idx)
    ref.assert_within(w, o_w, tol, "weights")
    np.testing.assert_array_equal(counts.cpu().numpy(),
                                  np.bincount(o_idx.reshape(-1), minlength=logits.shape[1]))


# groups of 2, 5 (through shared memory) and 32 experts (a register of the warp each)
@pytest.mark.parametrize("E,G,M", [(64, 32, 9), (60, 12, 5), (256, 8, 3)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("B", [1.0, 1000.0, 1e6])
def test_biases_that_cancel_in_a_group(moe, E, G, M, score, B):
    """A group's two best keys have biases of B and -B (the others' are lower still): their sum is of
    the scores' size, its fp32 error of the biases'."""
    S = E // G
    g = torch.Generator().manual_seed(E + int(B))
    logits = 1e-3 * torch.randn(600, E, generator=g)
    bias = torch.full((G, S), -4 * B)
    bias[:, 0], bias[:, -1] = B, -B
    check(moe, logits, M, bias.reshape(-1), score=score, n_group=G, topk_group=M)


@pytest.mark.parametrize("E,G,M", [(64, 32, 9), (60, 12, 5), (256, 8, 3)])
def test_one_group_of_large_biases_among_ordinary_ones(moe, E, G, M):
    """Biases that cancel in one group do not hide the borders of the others; a finite bias that
    disables an expert does not make its group uncertain."""
    S = E // G
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(600, E, generator=g)
    bias = 0.1 * torch.randn(G, S, generator=g)
    bias[1] = -1e30
    bias[1, 0], bias[1, -1] = 3e4, -3e4
    bias[2, 0] = -1e9
    bias[3] = -3e38  # (two of them are past the largest number)
    check(moe, logits, M, bias.reshape(-1), score="sigmoid", n_group=G, topk_group=M)


@pytest.mark.parametrize("E,G,M", [(64, 8, 3), (256, 8, 3), (512, 4, 2)])
@pytest.mark.parametrize("far", [80.0, 86.0, 87.0, 90.0, 101.0])
def test_softmax_scores_below_the_smallest_normal_number(moe, E, G, M, far):
    """Without a bias: the groups at the border have scores of e^-far / (experts in group 0)."""
    S = E // G
    g = torch.Generator().manual_seed(E + int(far))
    logits = -far - 1.5 * torch.rand(400, E, generator=g)
    logits[:, :S] = 0.0
    check(moe, logits, 10, None, score="softmax", n_group=G, topk_group=M)


@pytest.mark.parametrize("far", [85.0, 87.0, 88.0, 100.0])
def test_sigmoid_scores_below_the_smallest_normal_number(moe, far):
    g = torch.Generator().manual_seed(int(far))
    logits = -far - 1.5 * torch.rand(400, 64, generator=g)
    logits[:, :8] = 0.0
    check(moe, logits, 10, None, score="sigmoid", n_group=8, topk_group=3)
