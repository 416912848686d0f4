"""Weights of experts that a bias or a group limit selects far below the largest scores: a weight is
as exact as an fp32 number of its size, however small it is beside the others."""
import numpy as np
import pytest
import torch

import int8_ref as ref

pytestmark = pytest.mark.gpu


def check(moe, logits, K, bias, **rule):
    idx, w, _ = moe.route_logits(logits.cuda(), K, select_bias=None if bias is None else bias.cuda(), **rule)
    o_idx, o_w, tol = ref.route(logits, K, bias=bias, **rule)
    np.testing.assert_array_equal(idx.cpu().numpy(), o_idx)
    ref.assert_within(w, o_w, tol, "weights")
    return o_w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [-1.0, -10.0, -16.0, -18.0, -30.0, -60.0, -67.0, -70.0, -90.0, -300.0])
@pytest.mark.parametrize("renorm", [True, False])
def test_selected_scores_over_many_magnitudes(moe, score, best, renorm):
    """The bias selects experts 8 to 15, whose logits spread over 85 below `best`; expert 0 is at 0."""
    g = torch.Generator().manual_seed(int(-best))
    logits = torch.randn(200, 32, generator=g)
    logits[:, 0] = 0.0
    logits[:, 8:16] = best - torch.linspace(0, 85, 8) - torch.rand(200, 8, generator=g)
    bias = torch.zeros(32)
    bias[8:16] = 10.0 + 0.5 * torch.arange(8)  # (far apart: the selection is not the point here)
    w = check(moe, logits, 8, bias, score=score, n_group=1, topk_group=1, group_top=1, renorm=renorm)
    if renorm:
        assert (w > 1e-38).all() and w.min() < 1e-30


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,M", [(60, 30, 25), (32, 16, 6), (256, 8, 1)])
def test_wide_logits_and_large_biases(moe, score, E, G, M):
    g = torch.Generator().manual_seed(E)
    logits, bias = 30 * torch.randn(300, E, generator=g), 100 * torch.randn(E, generator=g)
    check(moe, logits, 7, bias, score=score, n_group=G, topk_group=M, group_top=2)
