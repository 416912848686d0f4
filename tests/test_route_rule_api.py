"""What a route_rule(...) is refused with, on the CPU: the rule holds a bare device pointer, so
its bias has to be where, and as long as, the kernel that reads it expects."""
import pytest
import torch

import top_routing_grouped_03_b200 as moe
from top_routing_grouped_03_b200 import build as moe_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.lib()


def weights(E, D=256, f=128):
    z = torch.zeros
    return z(E, D).bfloat16(), z(E, 2 * f, D).bfloat16(), z(E, D, f).bfloat16()


def test_a_bias_in_host_memory_is_refused():
    with pytest.raises(ValueError):
        moe.route_rule(8, 2, select_bias=torch.zeros(8))
    with pytest.raises(TypeError):
        moe.route_rule(8, 2, select_bias=torch.zeros(8, dtype=torch.float64))


def test_a_bias_of_another_length_is_refused():
    for shape in ((7,), (9,), (8, 1), ()):
        with pytest.raises(moe.MoEError):
            moe.route_rule(8, 2, select_bias=torch.zeros(shape))


def test_groups_that_hold_fewer_than_k_experts_are_refused():
    with pytest.raises(moe.MoEError):
        moe.route_rule(64, 9, n_group=8, topk_group=1)
    with pytest.raises(moe.MoEError):
        moe.route_rule(8, 9)
    assert moe.route_rule(64, 8, n_group=8, topk_group=1).topk_group == 1


def test_a_rule_for_another_number_of_experts_is_refused():
    w_router, gu, dn = weights(16)
    x = torch.zeros(4, 256).bfloat16()
    for E in (8, 32):
        rule = moe.route_rule(E, 2)
        with pytest.raises(moe.MoEError):
            moe.route(x, w_router, 2, rule=rule)
        with pytest.raises(moe.MoEError):
            moe.MoELayer(w_router, gu, dn, 2, rule=rule)
        layer = moe.MoELayer(w_router, gu, dn, 2, rule=moe.route_rule(16, 2))
        layer.rule = rule
        with pytest.raises(moe.MoEError):
            layer(x)


def test_a_bias_on_another_device_is_refused():
    """(The devices are those of the rule and of the weights: no launch is reached.)"""
    w_router, gu, dn = weights(16)
    x = torch.zeros(4, 256).bfloat16()
    rule = moe.route_rule(16, 2)
    rule.device = 1  # as route_rule sets it for a bias on cuda:1
    with pytest.raises(ValueError, match="cuda:1"):
        moe.route(x, w_router, 2, rule=rule)
    with pytest.raises(ValueError, match="cuda:1"):
        moe.MoELayer(w_router, gu, dn, 2, rule=rule)


def test_a_workspace_off_its_alignment_is_refused():
    import ctypes
    p = ctypes.c_void_p
    rule = moe.route_rule(128, 2)
    for T in (4, 300):  # CUDA-core and tensor-core logits
        for off, code in ((4, -3), (8, -3)):
            assert moe.lib().moe_route_rule_ex(p(0x10000), p(0x10000), None, None, T, 256, 128, 2, rule, p(0x10000),
                                               p(0x10000), p(0x10000), None, p(0x10000 + off), 1 << 40, None) == code
