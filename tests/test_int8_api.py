"""Refusals of the routing rules and the 8-bit integer entry points, on the CPU: every one
returns before anything is launched."""
import ctypes

import pytest
import torch

import top_routing_grouped_03_b200 as moe
from top_routing_grouped_03_b200 import build as moe_build

ARG, UNSUP, ALIGN, WS = -1, -2, -3, -6
A = 0x10000  # an aligned address that is never dereferenced


def ptr(a=A):
    return ctypes.c_void_p(a)


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.lib()


def rule(score=0, n_group=1, topk_group=1, group_top=1, renorm=1, scale=1.0):
    return moe.RouteRule(score, None, n_group, topk_group, group_top, renorm, scale)


@pytest.mark.parametrize("E,K,r,code", [
    (64, 4, rule(score=2), ARG), (64, 4, rule(n_group=0), ARG), (64, 4, rule(n_group=7), ARG),
    (64, 4, rule(n_group=8, topk_group=0), ARG), (64, 4, rule(n_group=8, topk_group=9), ARG),
    (64, 9, rule(n_group=8, topk_group=1), ARG), (64, 4, rule(n_group=64, topk_group=4), UNSUP),
    (64, 4, rule(group_top=3), ARG), (64, 4, rule(group_top=0), ARG),
    (64, 4, rule(scale=float("nan")), ARG), (64, 4, rule(scale=float("inf")), ARG),
    (513, 4, rule(), UNSUP), (64, 17, rule(), UNSUP), (3, 4, rule(), UNSUP), (0, 1, rule(), ARG)])
def test_rules_refused(lib, E, K, r, code):
    assert lib.moe_route_logits(ptr(), 0, 4, E, K, r, ptr(), ptr(), ptr(), None) == code
    assert lib.moe_route_rule_ex(ptr(), ptr(), None, None, 4, 128, E, K, r, ptr(), ptr(), ptr(), None,
                                 ptr(), 1 << 40, None) == code
    p = moe.LayerParams(ptr(), ptr(), None, ptr(), ptr(), None, None, None, 4, 128, E, K, 128)
    assert lib.moe_layer_forward_ex(p, r, None, ptr(), ptr(), 1 << 40, None) == code


def test_route_logits_refused(lib):
    f = lib.moe_route_logits
    assert f(ptr(), 0, 4, 64, 4, None, ptr(), ptr(), ptr(), None) == ARG
    assert f(ptr(), 2, 4, 64, 4, rule(), ptr(), ptr(), ptr(), None) == ARG
    assert f(None, 0, 4, 64, 4, rule(), ptr(), ptr(), ptr(), None) == ARG
    assert f(ptr(), 0, 4, 64, 4, rule(), None, ptr(), ptr(), None) == ARG
    assert f(ptr(), 0, 4, 64, 4, rule(), ptr(), None, ptr(), None) == ARG
    assert f(ptr(), 0, -1, 64, 4, rule(), ptr(), ptr(), ptr(), None) == ARG
    g = lib.moe_route_rule_ex
    ok = [ptr(), ptr(), None, None, 4, 128, 64, 4, rule(), ptr(), ptr(), ptr(), None, ptr(), 1 << 40, None]
    for i, v, code in ((1, None, ARG), (0, None, ARG), (0, ptr(A + 2), ALIGN), (3, ptr(), ARG),
                       (13, None, WS), (14, 100, WS), (5, 100, UNSUP), (8, None, ARG)):
        a = list(ok)
        a[i] = v
        assert g(*a) == code, (i, v)


def test_quantize_refused(lib):
    f = lib.moe_quantize_rows
    assert f(ptr(), 4, 40, ptr(), ptr(), None) == UNSUP
    assert f(ptr(), -1, 32, ptr(), ptr(), None) == ARG
    assert f(ptr(), 4, 0, ptr(), ptr(), None) == ARG
    assert f(ptr(), 1 << 31, 32, ptr(), ptr(), None) == UNSUP
    assert f(ptr(A + 8), 4, 32, ptr(), ptr(), None) == ALIGN
    assert f(None, 4, 32, ptr(), ptr(), None) == ARG
    assert f(None, 0, 32, None, None, None) == 0


def test_int8_matmul_refused(lib):
    assert lib.moe_int8_workspace_size(8, 64, 64) == 0  # a handful of tokens needs none
    n = lib.moe_int8_workspace_size(40, 64, 64)
    assert n > 0 and n % 256 == 0 and lib.moe_int8_workspace_size(4, 64, 32768) > 0
    for bad in ((40, 60, 64), (40, 64, 60), (-1, 64, 64), (40, 0, 64), (40, 64, 65552), (40, (1 << 20) + 8, 64)):
        assert lib.moe_int8_workspace_size(*bad) == 0, bad
    mm = [ptr(), ptr(), ptr(), ptr(), 40, 64, 64, ptr(), ptr(), n, None]
    ln = [ptr(), ptr(), ptr(), 40, 64, 64, ptr(), ptr(), n, None]
    for f, ok, cases in (
            (lib.moe_int8_matmul, mm, ((0, None, ARG), (1, None, ARG), (2, None, ARG), (3, None, ARG),
                                       (7, None, ARG), (8, None, WS), (9, n - 1, WS), (5, 60, UNSUP),
                                       (6, 24, UNSUP), (0, ptr(A + 8), ALIGN), (3, ptr(A + 4), ALIGN),
                                       (8, ptr(A + 16), ALIGN), (4, -1, ARG))),
            (lib.moe_int8_linear, ln, ((0, None, ARG), (1, None, ARG), (2, None, ARG), (6, None, ARG),
                                       (7, None, WS), (8, n - 1, WS), (4, 60, UNSUP), (5, 24, UNSUP),
                                       (0, ptr(A + 8), ALIGN), (2, ptr(A + 4), ALIGN), (3, -1, ARG)))):
        for i, v, code in cases:
            a = list(ok)
            a[i] = v
            assert f(*a) == code, (f, i, v)


def test_experts_int8_refused(lib):
    n = lib.moe_experts_int8_workspace_size(4, 256, 8, 2, 128, 0)
    assert 0 < n < lib.moe_experts_int8_workspace_size(4, 256, 8, 2, 128, 1)
    assert lib.moe_experts_int8_workspace_size(4, 250, 8, 2, 128, 0) == 0
    assert lib.moe_experts_int8_workspace_size(1 << 21, 8192, 8, 2, 128, 0) == 0

    def call(out=ptr(), ws=ptr(), size=n, **change):
        p = moe.Int8Experts(*[ptr()] * 11, None, 4, 256, 8, 2, 128, 0)
        for k, v in change.items():
            setattr(p, k, v)
        return lib.moe_experts_int8(p, out, ws, size, None)

    assert lib.moe_experts_int8(None, ptr(), ptr(), n, None) == ARG
    for name in ("xq", "x_scale", "expert_offsets", "sorted_token", "sorted_w", "slot_to_row", "w_gate_up",
                 "gate_up_scale", "w_down", "down_scale"):
        assert call(**{name: None}) == ARG, name
    for name in ("xq", "w_gate_up", "gate_up_scale", "w_down", "down_scale", "residual"):
        assert call(**{name: ptr(A + 8)}) == ALIGN, name
    big = lib.moe_experts_int8_workspace_size(4, 256, 8, 2, 128, 1)
    assert call(size=big, flags=1, topk_w=None) == ARG and call(size=big, flags=1, slot_to_row=None) == ARG
    assert call(out=None) == ARG and call(out=ptr(A + 8)) == ALIGN
    assert call(ws=None) == WS and call(size=n - 1) == WS and call(ws=ptr(A + 16)) == ALIGN
    assert call(D=200) == UNSUP and call(f=200) == UNSUP and call(K=9) == UNSUP and call(E=600) == UNSUP
    assert call(T=-1) == ARG


def test_layer_ex_refused(lib):
    size = lib.moe_layer_ex_workspace_size(4, 256, 8, 2, 128, 0, 0, 1)
    assert size > 0
    assert lib.moe_layer_ex_workspace_size(4, 256, 8, 2, 128, 0, 0, 0) == moe.workspace_size(4, 256, 8, 2, 128)
    assert lib.moe_layer_ex_workspace_size(4, 250, 8, 2, 128, 0, 0, 1) == 0

    def call(weights=None, r=None, out=ptr(), ws=ptr(), n=size, **change):
        p = moe.LayerParams(ptr(), ptr(), None, None, None, None, None, None, 4, 256, 8, 2, 128)
        for k, v in change.items():
            setattr(p, k, v)
        w = moe.Int8Weights(*[ptr()] * 4)
        for k, v in (weights or {}).items():
            setattr(w, k, v)
        return lib.moe_layer_forward_ex(p, r, w, out, ws, n, None)

    assert lib.moe_layer_forward_ex(None, None, None, ptr(), ptr(), size, None) == ARG
    for name in ("w_gate_up", "w_down", "w_shared_gate_up", "w_shared_down", "step_events"):
        assert call(**{name: ptr()}) == ARG, name  # bf16 weights beside the 8-bit ones
    assert call(w_router=None) == ARG and call(x=None) == ARG and call(out=None) == ARG
    for name in ("gate_up", "gate_up_scale", "down", "down_scale"):
        assert call({name: None}) == ARG and call({name: ptr(A + 4)}) == ALIGN, name
    assert call({"shared_down": ptr()}) == ARG and call(w_shared_gate=ptr()) == ARG and call(f_s=128) == ARG
    assert call(score_mode=5) == ARG and call(capacity_factor=-1.0) == ARG
    assert call(n=size - 1) == WS and call(ws=None) == WS and call(ws=ptr(A + 16)) == ALIGN
    assert call(r=rule(), score_mode=1) == ARG and call(r=rule(), select_bias=ptr()) == ARG
    assert call(r=rule(), flags=2) == ARG
    assert call(r=rule(n_group=3)) == ARG


def test_binding_refuses_before_launch(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, s = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    for call in (lambda: moe.route_logits(torch.zeros(4, 64), 4), lambda: moe.quantize_rows(x),
                 lambda: moe.int8_linear(x, w, s), lambda: moe.int8_matmul(w, s, w, s)):
        with pytest.raises(ValueError):  # no CUDA tensors
            call()
    with pytest.raises(moe.MoEError):
        moe.route_rule(64, 4, select_bias=torch.zeros(63))
