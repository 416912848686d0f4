"""The launch plan of a layer whose routing is a rule's: on the CPU by the host's count, on the GPU
against the launches of a call."""
import ctypes

import pytest
import torch

import top_routing_grouped_03_b200 as moe
from top_routing_grouped_03_b200 import build as moe_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.lib()


def plan(T, E, K, f_s=0, rule=None, flags=0, D=256, f=128):
    """(steps, launches) by the library, for a layer that is never run."""
    p = moe.LayerParams()
    p.x = p.w_router = p.w_gate_up = p.w_down = 0x10000
    if f_s:
        p.w_shared_gate = p.w_shared_gate_up = p.w_shared_down = 0x10000
    p.T, p.D, p.E, p.K, p.f, p.f_s, p.flags = T, D, E, K, f, f_s, flags
    mask, n = ctypes.c_uint(0), ctypes.c_int(0)
    rc = moe.lib().moe_layer_plan_ex(p, rule, ctypes.byref(mask), ctypes.byref(n))
    return rc, {s for i, s in enumerate(moe.STEP_EVENT_NAMES) if mask.value >> i & 1}, n.value


@pytest.mark.parametrize("f_s", [0, 128])
def test_a_rule_adds_its_launches(f_s):
    rule = moe.route_rule(16, 2, n_group=4, topk_group=2)
    rc, steps, n = plan(64, 16, 2, f_s)
    assert rc == 0 and plan(64, 16, 2, f_s, rule) == (0, steps, n + 1 + (f_s > 0))
    # tensor-core logits: the rule's kernel in the place of the plain selection
    rule = moe.route_rule(128, 2, n_group=4, topk_group=2)
    rc, steps, n = plan(300, 128, 2, f_s)
    assert rc == 0 and plan(300, 128, 2, f_s, rule) == (0, steps, n + (f_s > 0))
    assert plan(0, 128, 2, f_s, rule) == (0, set(), 0)


def test_refused_as_the_call_is():
    assert plan(64, 16, 2, rule=moe.route_rule(16, 2), flags=moe.MOE_FLAG_BF16_WEIGHTS)[0] == -1
    assert plan(64, 16, 2, rule=moe.RouteRule(0, None, 3, 1, 1, 1, 1.0))[0] == -1
    assert plan(64, 600, 2, rule=moe.route_rule(600, 2))[0] == -2
    assert moe.lib().moe_layer_plan_ex(None, None, None, None) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(1, 16), (64, 16), (300, 128), (600, 4)])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("ruled", [False, True])
def test_plan_counts_the_launches_of_a_call(T, E, shared, ruled):
    g = torch.Generator().manual_seed(T)

    def r(*s):
        return (torch.randn(*s, generator=g) / 16).bfloat16().cuda()

    extra = dict(w_shared_gate=r(256), w_shared_gate_up=r(256, 256), w_shared_down=r(256, 128)) if shared else {}
    rule = moe.route_rule(E, 2, "sigmoid", n_group=2, topk_group=1) if ruled else None
    layer = moe.MoELayer(r(E, 256), r(E, 256, 256), r(E, 256, 128), 2, rule=rule, **extra)
    x = r(T, 256)
    layer(x)
    before = moe.launch_count()
    layer(x)
    steps, n = layer.plan(T)
    assert moe.launch_count() - before == n and {"router", "permute", "gate_up", "down"} <= set(steps)
