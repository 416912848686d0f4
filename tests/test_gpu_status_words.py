"""The status word of a workspace tells about the call that used it, not about what the memory
held before, whichever kernels the sizes choose."""
import pytest
import torch

import int8_ref as ref

pytestmark = pytest.mark.gpu


def dirty(n):
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


# a handful of rows; weights on M; one-CTA tiles; CTA pairs
@pytest.mark.parametrize("T,E", [(3, 8), (12, 8), (40, 4), (600, 4)])
def test_experts_int8(moe, T, E):
    D, f, K = 256, 128, 2
    g = torch.Generator().manual_seed(T)
    gu, gus, dn, dns = (torch.stack(v).cuda() for v in zip(
        *[ref.channels(2 * f, D, g) + ref.channels(D, f, g) for _ in range(E)]))
    idx = torch.argsort(torch.rand(T, E, generator=g), dim=1)[:, :K].int().cuda().contiguous()
    w = torch.rand(T, K, generator=g).cuda()
    perm = moe.permute(idx, w, torch.bincount(idx.reshape(-1), minlength=E).int(), E)
    xq, xs = moe.quantize_rows(torch.randn(T, D, generator=g).bfloat16().cuda())
    ws = dirty(moe.lib().moe_experts_int8_workspace_size(T, D, E, K, f, 0))
    y = moe.experts_int8(xq, xs, w, perm, gu, gus, dn, dns, workspace=ws)
    assert moe.read_device_status(ws) == 0
    assert torch.equal(torch.isfinite(y), torch.ones_like(y, dtype=torch.bool))


@pytest.mark.parametrize("T,E", [(5, 64), (300, 128)])  # CUDA-core and tensor-core logits
@pytest.mark.parametrize("with_rule", [False, True])
def test_route(moe, T, E, with_rule):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, 256, generator=g).bfloat16().cuda()
    w = torch.randn(E, 256, generator=g).bfloat16().cuda()
    ws = dirty(moe.workspace_size(T, 256, E, 4, 128))
    moe.route(x, w, 4, workspace=ws, rule=moe.route_rule(E, 4, n_group=4, topk_group=2) if with_rule else None)
    assert moe.read_device_status(ws) == 0


@pytest.mark.parametrize("T", [40, 300])
def test_int8_products(moe, T):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, 256, generator=g).bfloat16().cuda()
    wq, s = (t.cuda() for t in ref.channels(264, 256, g))
    ws = dirty(moe.lib().moe_int8_workspace_size(T, 264, 256))
    y = moe.int8_linear(x, wq, s, workspace=ws)
    assert moe.read_device_status(ws) == 0
    ws.fill_(255)
    assert torch.equal(moe.int8_matmul(*moe.quantize_rows(x), wq, s, workspace=ws), y)
    assert moe.read_device_status(ws) == 0


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("T", [2, 64])
def test_a_layer_keeps_what_its_permutation_reported(moe, int8, T):
    """(No error here: the word is 0 from a dirty workspace, with few rows too.)"""
    g = torch.Generator().manual_seed(T)
    r = lambda *s: (torch.randn(*s, generator=g) / 16).bfloat16().cuda()
    layer = (moe.Int8MoELayer if int8 else moe.MoELayer)(r(8, 256), r(8, 256, 256), r(8, 256, 128), 2,
                                                         rule=moe.route_rule(8, 2, n_group=2, topk_group=1))
    x = r(T, 256)
    layer.workspace(T).fill_(255)
    layer(x)
    assert layer.device_status() == 0
