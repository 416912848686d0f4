"""A workspace stays in place for as long as a captured graph, or work on another stream, uses it."""
import weakref

import pytest
import torch

pytestmark = pytest.mark.gpu


def make(moe, int8):
    g = torch.Generator().manual_seed(3)

    def r(*s):
        return (torch.randn(*s, generator=g) / 16).bfloat16().cuda()

    cls = moe.Int8MoELayer if int8 else moe.MoELayer
    return cls(r(16, 256), r(16, 256, 256), r(16, 256, 128), 2, deterministic=True), r


@pytest.mark.parametrize("int8", [False, True])
def test_a_captured_call_keeps_its_workspace(moe, int8):
    layer, r = make(moe, int8)
    x, big = r(24, 256), r(3000, 256)
    want = layer(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer(x)
    old = weakref.ref(layer._ws)
    size = layer._ws.numel()
    layer(big)
    assert layer._ws is not old() and old() is not None
    # nobody else gets the memory that replays write to
    others = [torch.full((size,), 17, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(3):
        y.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all(bool((o == 17).all()) for o in others)
    # captured again, on the workspace of now: one more is kept, not one for every call
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        layer(x)
        layer(x)
    assert len(layer._captured_ws) == 2
    del g, g2


@pytest.mark.parametrize("int8", [False, True])
def test_a_workspace_in_use_on_another_stream_is_not_handed_on(moe, int8):
    layer, r = make(moe, int8)
    x, big = r(2000, 256), r(4000, 256)
    want = layer(x)
    side = torch.cuda.Stream()
    ptr, size = layer._ws.data_ptr(), layer._ws.numel()
    # memory for the larger workspace is at hand: taking it does not wait for the GPU
    other, _ = make(moe, int8)
    other.workspace(4000)
    del other
    torch.cuda.synchronize()
    ys = []
    with torch.cuda.stream(side):
        torch.cuda._sleep(500_000_000)  # (a quarter of a second) the call below is still to come when
    ys.append(layer(x, stream=side))    # the layer moves on
    layer.workspace(4000)
    held = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert held.data_ptr() != ptr
    torch.cuda.synchronize()
    assert torch.equal(ys[0], want)
    assert torch.equal(layer(big)[:1].isfinite(), torch.ones(1, 256, dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("ruled", [False, True])
def test_a_call_of_its_own_workspace_on_another_stream(moe, ruled, monkeypatch):
    """The workspaces that route and permute allocate for one call, dropped before it has run."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(2000, 256, generator=g).bfloat16().cuda()
    w = torch.randn(64, 256, generator=g).bfloat16().cuda()
    rule = moe.route_rule(64, 4, n_group=4, topk_group=2) if ruled else None
    want = moe.route(x, w, 4, rule=rule)
    perm = moe.permute(want[0], want[1], want[2], 64)
    lent, alloc = [], moe.alloc_workspace

    def spy(*a, **k):
        ws = alloc(*a, **k)
        lent.append((ws.data_ptr(), ws.numel()))
        return ws

    monkeypatch.setattr(moe, "alloc_workspace", spy)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(500_000_000)
    got = moe.route(x, w, 4, rule=rule, stream=side)
    got_perm = moe.permute(got[0], got[1], got[2], 64, stream=side)
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in lent]
    assert len(lent) == 2 and not {h.data_ptr() for h in held} & {p for p, _ in lent}
    torch.cuda.synchronize()
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(got_perm[k], perm[k]) for k in perm)
