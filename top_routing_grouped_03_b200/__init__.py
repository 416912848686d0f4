"""top_routing_grouped_03_b200 -- one top-k MoE SwiGLU FFN layer forward on a B200.

A thin ctypes binding over ``libmoe_b200.so`` (C ABI in ``include/moe_api.h``).  Every
step of the layer runs in the library's sm_100a kernels; this module only allocates
tensors with PyTorch, passes their device pointers and the current CUDA stream, and turns
status codes into exceptions.  There is no fallback: without the built library (or on a
machine without a CUDA device) the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_b200.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "moe_api.h")

MOE_FLAG_DETERMINISTIC = 1
MOE_FLAG_BF16_WEIGHTS = 2
SCORES = {"softmax": 0, "sigmoid": 1}

_lib = None


class MoEError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


class LayerParams(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("w_router", ctypes.c_void_p), ("logit_bias", ctypes.c_void_p),
        ("w_gate_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
        ("w_shared_gate", ctypes.c_void_p), ("w_shared_gate_up", ctypes.c_void_p),
        ("w_shared_down", ctypes.c_void_p),
        ("T", ctypes.c_int), ("D", ctypes.c_int), ("E", ctypes.c_int), ("K", ctypes.c_int),
        ("f", ctypes.c_int), ("f_s", ctypes.c_int), ("flags", ctypes.c_uint),
        ("topk_idx_out", ctypes.c_void_p), ("topk_w_out", ctypes.c_void_p),
        ("expert_counts_out", ctypes.c_void_p), ("step_events", ctypes.c_void_p),
        ("score_mode", ctypes.c_int), ("select_bias", ctypes.c_void_p),
        ("residual", ctypes.c_void_p),
        ("capacity_factor", ctypes.c_float), ("min_capacity", ctypes.c_int),
    ]


class RouteRule(ctypes.Structure):
    """moe_route_rule."""
    _fields_ = [
        ("score_mode", ctypes.c_int), ("select_bias", ctypes.c_void_p),
        ("n_group", ctypes.c_int), ("topk_group", ctypes.c_int), ("group_top", ctypes.c_int),
        ("renorm", ctypes.c_int), ("scale", ctypes.c_float),
    ]
    # set by route_rule(): the bias that select_bias points to, its CUDA device and its length
    keep = device = E = None


class Int8Experts(ctypes.Structure):
    """moe_int8_experts."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "xq", "x_scale", "expert_offsets", "sorted_token", "sorted_w", "slot_to_row", "topk_w",
        "w_gate_up", "gate_up_scale", "w_down", "down_scale", "residual")] + \
        [(n, ctypes.c_int) for n in ("T", "D", "E", "K", "f")] + [("flags", ctypes.c_uint)]


class Int8Weights(ctypes.Structure):
    """moe_int8_weights."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "gate_up", "gate_up_scale", "down", "down_scale", "shared_gate_up", "shared_gate_up_scale",
        "shared_down", "shared_down_scale")]


# Step boundaries recorded by moe_layer_forward when step_events is given.
STEP_EVENT_NAMES = ("start", "router", "permute", "gate_up", "down", "shared", "combine",
                    "end")
NUM_STEP_EVENTS = len(STEP_EVENT_NAMES)


def lib() -> ctypes.CDLL:
    """Load the C library (built in-tree by ``build.build()`` / ``__graft_entry__.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m top_routing_grouped_03_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_status_string.argtypes = [I]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_version.argtypes = []
        L.moe_version.restype = I
        L.moe_workspace_size.argtypes = [I, I, I, I, I, I]
        L.moe_workspace_size.restype = Z
        L.moe_route.argtypes = [P, P, P, P, I, I, I, I, P, P, P, P, P, Z, P]
        L.moe_route.restype = I
        L.moe_route_ex.argtypes = [P, P, P, P, I, I, I, I, I, P, ctypes.c_uint, P, P, P, P, P,
                                   Z, P]
        L.moe_route_ex.restype = I
        L.moe_permute.argtypes = [P, P, P, I, I, I, P, P, P, P, P, P]
        L.moe_permute.restype = I
        L.moe_permute_ex.argtypes = [P, P, P, I, I, I, ctypes.c_longlong, P, P, P, P, P, P]
        L.moe_permute_ex.restype = I
        L.moe_expert_capacity.argtypes = [I, I, I, ctypes.c_float, I]
        L.moe_expert_capacity.restype = ctypes.c_longlong
        L.moe_grouped_swiglu.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P, P, P, Z, P]
        L.moe_grouped_swiglu.restype = I
        L.moe_combine.argtypes = [P, P, P, P, P, P, I, I, I, P, P]
        L.moe_combine.restype = I
        L.moe_layer_forward.argtypes = [ctypes.POINTER(LayerParams), P, P, Z, P]
        L.moe_layer_forward.restype = I
        L.moe_read_device_status.argtypes = [P, P]
        L.moe_read_device_status.restype = I
        L.moe_route_noalloc.argtypes = [P, P, P, P, I, I, I, I, P, P, P, P, P]
        L.moe_route_noalloc.restype = I
        L.moe_launch_count.argtypes = []
        L.moe_launch_count.restype = ctypes.c_ulonglong
        L.moe_ep_dispatch_rows.argtypes = [P, P, I, I, P, P]
        L.moe_ep_dispatch_rows.restype = I
        L.moe_ep_recv_layout.argtypes = [P, I, I, I, P, P, P, P]
        L.moe_ep_recv_layout.restype = I
        L.moe_ep_return_rows.argtypes = [P, P, I, I, P, P]
        L.moe_ep_return_rows.restype = I
        L.moe_layer_plan.argtypes = [ctypes.POINTER(LayerParams), P, P]
        L.moe_layer_plan.restype = I
        L.moe_set_grid_wait_budget_ns.argtypes = [ctypes.c_ulonglong]
        L.moe_set_grid_wait_budget_ns.restype = ctypes.c_ulonglong
        RP = ctypes.POINTER(RouteRule)
        L.moe_route_logits.argtypes = [P, I, I, I, I, RP, P, P, P, P]
        L.moe_route_logits.restype = I
        L.moe_route_rule_ex.argtypes = [P, P, P, P, I, I, I, I, RP, P, P, P, P, P, Z, P]
        L.moe_route_rule_ex.restype = I
        L.moe_quantize_rows.argtypes = [P, ctypes.c_longlong, I, P, P, P]
        L.moe_quantize_rows.restype = I
        L.moe_int8_workspace_size.argtypes = [I, I, I]
        L.moe_int8_workspace_size.restype = Z
        L.moe_int8_matmul.argtypes = [P, P, P, P, I, I, I, P, P, Z, P]
        L.moe_int8_matmul.restype = I
        L.moe_int8_linear.argtypes = [P, P, P, I, I, I, P, P, Z, P]
        L.moe_int8_linear.restype = I
        L.moe_experts_int8_workspace_size.argtypes = [I, I, I, I, I, ctypes.c_uint]
        L.moe_experts_int8_workspace_size.restype = Z
        L.moe_experts_int8.argtypes = [ctypes.POINTER(Int8Experts), P, P, Z, P]
        L.moe_experts_int8.restype = I
        L.moe_layer_ex_workspace_size.argtypes = [I, I, I, I, I, I, ctypes.c_uint, I]
        L.moe_layer_ex_workspace_size.restype = Z
        L.moe_layer_forward_ex.argtypes = [ctypes.POINTER(LayerParams), RP,
                                           ctypes.POINTER(Int8Weights), P, P, Z, P]
        L.moe_layer_forward_ex.restype = I
        L.moe_layer_plan_ex.argtypes = [ctypes.POINTER(LayerParams), RP, P, P]
        L.moe_layer_plan_ex.restype = I
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().moe_status_string(int(code)).decode()


def version() -> int:
    return lib().moe_version()


def _check(rc: int, what: str):
    if rc != 0:
        raise MoEError(rc, what)


BF16, F32, I32, U8, I8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.int8


def _p(t: Optional[torch.Tensor], dtype: Optional[torch.dtype] = None):
    """Device pointer of a contiguous CUDA tensor (None -> NULL), of the element type the
    C ABI reads there when ``dtype`` is given."""
    if t is None:
        return None
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"expected a {dtype} tensor, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def workspace_size(T: int, D: int, E: int, K: int, f: int, f_s: int = 0) -> int:
    return int(lib().moe_workspace_size(T, D, E, K, f, f_s))


def alloc_workspace(T, D, E, K, f, f_s=0, device=None) -> torch.Tensor:
    n = workspace_size(T, D, E, K, f, f_s)
    if n == 0:
        raise MoEError(-2, "moe_workspace_size")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    ws[:256].zero_()  # the device status word starts clear
    return ws


def _lend(workspace, stream):
    """A workspace that is dropped when the call returns stays out of other hands until ``stream``, if
    it is not the one the workspace was allocated on, has got past the call."""
    if stream is not None:
        workspace.record_stream(stream)


def route(x, w_router, K, logit_bias=None, w_shared_gate=None, workspace=None, stream=None,
          score="softmax", select_bias=None, bf16_weights=False, rule=None):
    """Router step.  Returns (topk_idx [T,K] int32, topk_w [T,K] f32, expert_counts [E]
    int32, shared_gate [T] f32 or None).  score / select_bias / bf16_weights select the
    router variants of moe_route_ex; ``rule`` (a route_rule(...)) those of moe_route_rule_ex
    instead."""
    T, D = x.shape
    E = w_router.shape[0]
    dev = x.device
    _check_rule(rule, E, x)
    ws = workspace
    if ws is None:
        ws = alloc_workspace(T, D, E, K, 128, 0, dev)
        _lend(ws, stream)
    idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    w = torch.empty((T, K), dtype=torch.float32, device=dev)
    counts = torch.empty((E,), dtype=torch.int32, device=dev)
    sg = torch.empty((T,), dtype=torch.float32, device=dev) if w_shared_gate is not None else None
    if rule is not None:
        _need(score == "softmax" and select_bias is None and not bf16_weights,
              "route (a rule replaces score, select_bias and bf16_weights)")
        rc = lib().moe_route_rule_ex(_p(x, BF16), _p(w_router, BF16), _p(logit_bias, F32),
                                     _p(w_shared_gate, BF16), T, D, E, K, rule, _p(idx), _p(w),
                                     _p(counts), _p(sg), _p(ws, U8), ws.numel(), _stream(stream))
    elif score == "softmax" and select_bias is None and not bf16_weights:
        rc = lib().moe_route(_p(x, BF16), _p(w_router, BF16), _p(logit_bias, F32),
                             _p(w_shared_gate, BF16), T, D, E, K, _p(idx), _p(w), _p(counts),
                             _p(sg), _p(ws, U8), ws.numel(), _stream(stream))
    else:
        rc = lib().moe_route_ex(_p(x, BF16), _p(w_router, BF16), _p(logit_bias, F32),
                                _p(w_shared_gate, BF16), T, D, E, K, SCORES[score],
                                _p(select_bias, F32),
                                MOE_FLAG_BF16_WEIGHTS if bf16_weights else 0, _p(idx), _p(w),
                                _p(counts), _p(sg), _p(ws, U8), ws.numel(), _stream(stream))
    _check(rc, "moe_route")
    return idx, w, counts, sg


def route_noalloc(x, w_router, K, logit_bias=None, w_shared_gate=None, stream=None):
    """Router step with no workspace: the library's own 1 MiB device scratch is used (see
    moe_route_noalloc in moe_api.h for the size limit and the sharing rules).  Only the
    outputs are allocated here, by the caller's side of the binding."""
    T, D = x.shape
    E = w_router.shape[0]
    dev = x.device
    idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    w = torch.empty((T, K), dtype=torch.float32, device=dev)
    counts = torch.empty((E,), dtype=torch.int32, device=dev)
    sg = torch.empty((T,), dtype=torch.float32, device=dev) if w_shared_gate is not None else None
    rc = lib().moe_route_noalloc(_p(x, BF16), _p(w_router, BF16), _p(logit_bias, F32),
                                 _p(w_shared_gate, BF16), T, D, E, K, _p(idx), _p(w),
                                 _p(counts), _p(sg), _stream(stream))
    _check(rc, "moe_route_noalloc")
    return idx, w, counts, sg


def expert_capacity(T, K, E, capacity_factor, min_capacity=0) -> int:
    """Assignments per expert the layer keeps (moe_expert_capacity); -1: no capacity."""
    return int(lib().moe_expert_capacity(T, K, E, float(capacity_factor), int(min_capacity)))


def permute(topk_idx, topk_w, expert_counts, E, workspace=None, stream=None, capacity=None):
    """Permutation step.  Returns dict(offsets [E+1], sorted_token, sorted_w, slot_to_row).
    ``capacity``: keep each expert's first ``capacity`` entries (moe_permute_ex)."""
    T, K = topk_idx.shape
    dev = topk_idx.device
    off = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    st = torch.empty((T * K,), dtype=torch.int32, device=dev)
    sw = torch.empty((T * K,), dtype=torch.float32, device=dev) if topk_w is not None else None
    s2r = torch.empty((T * K,), dtype=torch.int32, device=dev)
    if workspace is None and T > 0:
        workspace = alloc_workspace(T, 128, E, K, 128, 0, dev)
        _lend(workspace, stream)
    cap = -1 if capacity is None else int(capacity)
    rc = lib().moe_permute_ex(_p(topk_idx, I32), _p(topk_w, F32), _p(expert_counts, I32), T, E,
                              K, cap, _p(off), _p(st), _p(sw), _p(s2r), _p(workspace, U8),
                              _stream(stream))
    _check(rc, "moe_permute_ex")
    return dict(offsets=off, sorted_token=st, sorted_w=sw, slot_to_row=s2r)


def grouped_swiglu(x, sorted_token, offsets, sorted_w, w_gate_up, w_down, rows,
                   out_acc=None, y_sorted=None, workspace=None, stream=None):
    """Grouped SwiGLU experts over the sorted rows; writes out_acc (+=) and/or y_sorted."""
    T, D = x.shape
    E, twof, _ = w_gate_up.shape
    f = twof // 2
    if workspace is None:
        Kr = max(1, -(-rows // max(T, 1)))
        workspace = alloc_workspace(max(T, 1), D, E, min(Kr, E, 16), f, 0, x.device)
        _lend(workspace, stream)
    rc = lib().moe_grouped_swiglu(_p(x, BF16), _p(sorted_token, I32), _p(offsets, I32),
                                  _p(sorted_w, F32), _p(w_gate_up, BF16), _p(w_down, BF16), T,
                                  rows, D, E, f, _p(y_sorted, F32), _p(out_acc, F32),
                                  _p(workspace, U8), workspace.numel(), _stream(stream))
    _check(rc, "moe_grouped_swiglu")


def combine(T, D, K, out=None, out_acc=None, y_sorted=None, slot_to_row=None, topk_w=None,
            shared_out=None, shared_gate=None, device=None, stream=None):
    dev = device or "cuda"
    out = out if out is not None else torch.empty((T, D), dtype=torch.bfloat16, device=dev)
    rc = lib().moe_combine(_p(out_acc, F32), _p(y_sorted, F32), _p(slot_to_row, I32),
                           _p(topk_w, F32), _p(shared_out, BF16), _p(shared_gate, F32), T, D, K,
                           _p(out, BF16), _stream(stream))
    _check(rc, "moe_combine")
    return out


def _need(ok: bool, what: str):
    if not ok:
        raise MoEError(-1, what)


_empty = torch.empty_strided  # (the call that costs the host least)
# torch's own, without the objects around them, which small calls notice; a torch without them, as
# one built for the CPU, takes the public ones
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _on_device_of(fn):
    """Runs fn with its first argument's device current and its ``stream`` (default: that
    device's current stream) as the current one, so that what fn allocates belongs to it."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if args and name not in kw:
            first = args[0]
        elif name in kw and not args:
            first = kw[name]
        else:
            return fn(*args, **kw)  # says what is wrong
        index = first.get_device()
        if index < 0:
            raise ValueError("expected a CUDA tensor")
        if stream is None and index == _get_device():
            return fn(*args, **kw)
        if stream is None:
            stream = torch.cuda.current_stream(index)
        if stream.device != first.device:
            raise ValueError(f"stream on {stream.device}, tensors on {first.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _q(t, dtype, index):
    """Address of a contiguous tensor of type ``dtype`` on CUDA device ``index`` (None -> NULL)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.is_cuda and t.get_device() != index:
        raise ValueError(f"expected a tensor on cuda:{index}, got one on {t.device}")
    return _p(t, dtype)  # says what is wrong


def _sizes(what, *sizes):
    """The C ABI takes these as 32-bit ints, and ctypes would hand over their low 32 bits.  (Calls
    that small batches make look at the bits of all first.)"""
    if max(sizes) > 0x7fffffff:
        raise MoEError(-2, f"{what} (a size of 2^31 or more)")


def route_rule(E, K, score="softmax", select_bias=None, n_group=1, topk_group=1, group_top=None,
               renorm=True, scale=1.0) -> RouteRule:
    """A moe_route_rule for routers of E experts (and K of them a token, which the groups that
    stay have to hold).  group_top defaults to 2 with a select_bias (a group is judged by its two
    best keys) and 1 without."""
    if select_bias is not None:
        _need(select_bias.shape == (E,), "route_rule (select_bias must be [E])")
    _sizes("route_rule", E, K, n_group, topk_group, 1 if group_top is None else group_top)
    if n_group > 0 and E % n_group == 0:
        _need(K <= topk_group * (E // n_group), "route_rule (K experts in the groups that stay)")
    if group_top is None:
        group_top = 1 if select_bias is None else 2
    rule = RouteRule(SCORES[score], _p(select_bias, F32), n_group, topk_group, group_top,
                     1 if renorm else 0, scale)
    rule.keep, rule.E = select_bias, E
    rule.device = None if select_bias is None else select_bias.get_device()
    return rule


def _check_rule(rule, E, on):
    """A rule's bias is as long as the router has experts, and on the device of tensor ``on``."""
    if rule is None:
        return
    _need(rule.E is None or rule.E == E, f"route_rule (made for {rule.E} experts, used with {E})")
    if rule.device is not None and rule.device != on.get_device():
        raise ValueError(f"route_rule: select_bias on cuda:{rule.device}, tensors on {on.device}")


@_on_device_of
def route_logits(logits, K, score="softmax", select_bias=None, n_group=1, topk_group=1,
                 group_top=None, renorm=True, scale=1.0):
    """Routing from given logits [T, E] (fp32 or bf16) by moe_route_logits: scores, a
    selection-only bias, the topk_group best of n_group expert groups, TopK, weights
    (renormalised, times scale).  Returns (topk_idx [T,K] int32, topk_w [T,K] f32,
    expert_counts [E] int32)."""
    _need(logits.dim() == 2, "route_logits (logits must be [T, E])")
    T, E = logits.shape
    dev = logits.get_device()
    if (T | E | K | n_group | topk_group) >> 31:
        _sizes("route_logits", T, E, K, n_group, topk_group)
    kind = 0 if logits.dtype is F32 else 1
    if select_bias is not None:
        _need(select_bias.numel() == E, "route_logits (select_bias must be [E])")
    if group_top is None:
        group_top = 1 if select_bias is None else 2
    rule = RouteRule(SCORES[score], _q(select_bias, F32, dev), n_group, topk_group, group_top,
                     1 if renorm else 0, scale)
    x = _q(logits, F32 if kind == 0 else BF16, dev)
    device = logits.device
    idx = _empty((T, K), (K, 1), dtype=I32, device=device)
    w = _empty((T, K), (K, 1), dtype=F32, device=device)
    counts = _empty((E,), (1,), dtype=I32, device=device)
    _check(lib().moe_route_logits(x, kind, T, E, K, rule, idx.data_ptr(), w.data_ptr(),
                                  counts.data_ptr(), _raw_stream(dev)), "moe_route_logits")
    return idx, w, counts


@_on_device_of
def quantize_rows(x):
    """Rows of x [..., C] bf16 as 8-bit integers: (q int8 like x, scale [...] f32) with
    x ~ q * scale (moe_quantize_rows)."""
    _need(x.dim() >= 1, "quantize_rows (x must have rows)")
    dev = x.get_device()
    p = _q(x, BF16, dev)
    shape, stride, device = x.shape, x.stride(), x.device  # (x is contiguous)
    cols = shape[-1]
    if cols >> 31:
        _sizes("quantize_rows", cols)
    q = _empty(shape, stride, dtype=I8, device=device)
    if len(shape) == 2:
        scale = _empty((shape[0],), (1,), dtype=F32, device=device)
    else:
        scale = torch.empty(shape[:-1], dtype=F32, device=device)
    _check(lib().moe_quantize_rows(p, scale.numel(), cols, q.data_ptr(), scale.data_ptr(),
                                   _raw_stream(dev)), "moe_quantize_rows")
    return q, scale


def _int8_buffers(x, T, N, K, out, workspace):
    if out is None:
        out = _empty((T, N), (N, 1), dtype=BF16, device=x.device)
    else:
        _need(out.shape == (T, N), "int8 product (out must be [T, N])")
    if workspace is not None:
        return out, workspace, workspace.numel()
    n = int(lib().moe_int8_workspace_size(T, N, K))  # 0: none needed, or an unsupported shape
    return out, _empty((n,), (1,), dtype=U8, device=x.device) if n else None, n


@_on_device_of
def int8_matmul(xq, x_scale, wq, w_scale, workspace=None, out=None):
    """out [T, N] bf16 = (xq wq^T) * x_scale[:, None] * w_scale[None, :] with xq [T, K] and
    wq [N, K] int8 (moe_int8_matmul)."""
    _need(xq.dim() == 2 and wq.dim() == 2 and xq.shape[1] == wq.shape[1],
          "int8_matmul (xq must be [T, K], wq [N, K])")
    (T, K), N, dev = xq.shape, wq.shape[0], xq.get_device()
    if (T | K | N) >> 31:
        _sizes("int8_matmul", T, K, N)
    _need(x_scale.shape == (T,) and w_scale.shape == (N,), "int8_matmul (one scale per row)")
    a = _q(xq, I8, dev), _q(x_scale, F32, dev), _q(wq, I8, dev), _q(w_scale, F32, dev)
    out, ws, n = _int8_buffers(xq, T, N, K, out, workspace)
    _check(lib().moe_int8_matmul(*a, T, N, K, _q(out, BF16, dev), _q(ws, U8, dev), n,
                                 _raw_stream(dev)), "moe_int8_matmul")
    return out


@_on_device_of
def int8_linear(x, wq, w_scale, workspace=None, out=None):
    """A linear layer in 8-bit integers: x [T, K] bf16 quantised per row, times wq [N, K] int8
    with w_scale [N]; returns [T, N] bf16 (moe_int8_linear).  A ``workspace`` of the caller's holds
    the status word that read_device_status reads (a handful of tokens uses none)."""
    _need(x.dim() == 2 and wq.dim() == 2 and x.shape[1] == wq.shape[1],
          "int8_linear (x must be [T, K], wq [N, K])")
    (T, K), N, dev = x.shape, wq.shape[0], x.get_device()
    if (T | K | N) >> 31:
        _sizes("int8_linear", T, K, N)
    _need(w_scale.shape == (N,), "int8_linear (one scale per weight row)")
    a = _q(x, BF16, dev), _q(wq, I8, dev), _q(w_scale, F32, dev)
    out, ws, n = _int8_buffers(x, T, N, K, out, workspace)
    _check(lib().moe_int8_linear(*a, T, N, K, _q(out, BF16, dev), _q(ws, U8, dev), n,
                                 _raw_stream(dev)), "moe_int8_linear")
    return out


@_on_device_of
def experts_int8(xq, x_scale, topk_w, perm, w_gate_up, gate_up_scale, w_down, down_scale,
                 residual=None, deterministic=False, workspace=None, out=None):
    """The routed SwiGLU experts in 8-bit integers (moe_experts_int8): tokens xq [T, D] int8 with
    x_scale [T] (quantize_rows), weights w_gate_up [E, 2f, D] and w_down [E, D, f] int8 with
    gate_up_scale [E, 2f] and down_scale [E, D], for the routing weights topk_w [T, K] and
    ``perm`` = permute(...).  Returns out [T, D] bf16 (+ residual).  Rows of ``perm`` are trusted:
    they must index the T tokens and the E experts.  A ``workspace`` of the caller's holds the
    status word that read_device_status reads."""
    _need(xq.dim() == 2 and w_down.dim() == 3 and topk_w.dim() == 2,
          "experts_int8 (xq [T, D], topk_w [T, K], w_gate_up [E, 2f, D], w_down [E, D, f])")
    T, D = xq.shape
    E, _, f = w_down.shape
    K, dev = topk_w.shape[1], xq.get_device()
    _need(topk_w.shape[0] == T and w_down.shape[1] == D and w_gate_up.shape == (E, 2 * f, D),
          "experts_int8 (weights and tokens of different shapes)")
    _need(x_scale.numel() == T and gate_up_scale.numel() == 2 * E * f and down_scale.numel() == E * D,
          "experts_int8 (one scale per row)")
    offsets, token, weight, row = (perm["offsets"], perm["sorted_token"], perm["sorted_w"],
                                   perm["slot_to_row"])
    n = T * K
    if (T | D | E | K | f) >> 31:
        _sizes("experts_int8", T, D, E, K, f)
    _need(offsets.numel() == E + 1 and token.numel() == n and weight.numel() == n
          and row.numel() == n, "experts_int8 (perm of another routing)")
    _need((out is None or out.shape == (T, D)) and (residual is None or residual.shape == (T, D)),
          "experts_int8 (out and residual must be [T, D])")
    flags = MOE_FLAG_DETERMINISTIC if deterministic else 0
    prm = Int8Experts(_q(xq, I8, dev), _q(x_scale, F32, dev), _q(offsets, I32, dev),
                      _q(token, I32, dev), _q(weight, F32, dev), _q(row, I32, dev),
                      _q(topk_w, F32, dev), _q(w_gate_up, I8, dev), _q(gate_up_scale, F32, dev),
                      _q(w_down, I8, dev), _q(down_scale, F32, dev), _q(residual, BF16, dev),
                      T, D, E, K, f, flags)
    if workspace is None:
        n = int(lib().moe_experts_int8_workspace_size(T, D, E, K, f, flags))
        if n == 0:
            raise MoEError(-2, "moe_experts_int8_workspace_size")
        workspace = _empty((n,), (1,), dtype=U8, device=xq.device)
    if out is None:
        out = _empty((T, D), (D, 1), dtype=BF16, device=xq.device)
    _check(lib().moe_experts_int8(prm, _q(out, BF16, dev), _q(workspace, U8, dev),
                                  workspace.numel(), _raw_stream(dev)), "moe_experts_int8")
    return out


def ep_dispatch_rows(x, sorted_token, rows, stream=None):
    """x_sorted [rows, D] bf16 = x[sorted_token[:rows]] (moe_ep_dispatch_rows)."""
    out = torch.empty((rows, x.shape[1]), dtype=BF16, device=x.device)
    _check(lib().moe_ep_dispatch_rows(_p(x, BF16), _p(sorted_token, I32), rows, x.shape[1],
                                      _p(out, BF16), _stream(stream)), "moe_ep_dispatch_rows")
    return out


def ep_recv_layout(recv_counts, n, workspace=None, stream=None):
    """(recv_offsets [El+1], recv_row [n]) from the received counts [G, El] (device int32)."""
    G, El = recv_counts.shape
    off = torch.empty((El + 1,), dtype=I32, device=recv_counts.device)
    row = torch.empty((n,), dtype=I32, device=recv_counts.device)
    _check(lib().moe_ep_recv_layout(_p(recv_counts, I32), G, El, n, _p(off), _p(row),
                                    _p(workspace, U8), _stream(stream)), "moe_ep_recv_layout")
    return off, row


def ep_return_rows(y, recv_row, stream=None):
    """y_ret [n, D] fp32 with y_ret[recv_row[j]] = y[j] (moe_ep_return_rows)."""
    n, D = y.shape
    out = torch.empty_like(y)
    _check(lib().moe_ep_return_rows(_p(y, F32), _p(recv_row, I32), n, D, _p(out, F32),
                                    _stream(stream)), "moe_ep_return_rows")
    return out


def launch_count() -> int:
    """Kernels launched by the library in this process so far."""
    return int(lib().moe_launch_count())


def set_grid_wait_budget_ns(ns: int) -> int:
    """Bound of the layer's grid-wide wait for later calls (moe_set_grid_wait_budget_ns);
    returns the previous bound."""
    return int(lib().moe_set_grid_wait_budget_ns(int(ns)))


def event_array(events):
    """ctypes array of raw cudaEvent_t handles of recorded ``torch.cuda.Event`` objects
    (None entries are not recorded by the layer)."""
    assert len(events) == NUM_STEP_EVENTS
    arr = (ctypes.c_void_p * NUM_STEP_EVENTS)()
    for i, e in enumerate(events):
        if e is None:
            arr[i] = None
            continue
        if not e.cuda_event:
            raise ValueError("record each event once before passing it (creates the handle)")
        arr[i] = e.cuda_event
    return arr


def read_device_status(workspace, stream=None) -> int:
    return int(lib().moe_read_device_status(_p(workspace), _stream(stream)))


class MoELayer:
    """One MoE layer with resident weights and a reusable workspace.

    ``layer(x)`` runs moe_layer_forward on the current stream and returns y [T, D] bf16.
    Calls share the layer's workspace, so they must not overlap on the GPU (one stream, or
    ordered by events), replays of captured calls included.  A larger batch replaces the
    workspace; the one that a captured call used stays with the layer.
    """

    def __init__(self, w_router, w_gate_up, w_down, K, logit_bias=None, w_shared_gate=None,
                 w_shared_gate_up=None, w_shared_down=None, deterministic=False,
                 score="softmax", select_bias=None, bf16_weights=False, capacity_factor=0.0,
                 min_capacity=0, rule=None):
        self.w_router, self.w_gate_up, self.w_down = w_router, w_gate_up, w_down
        self.logit_bias = logit_bias
        self.w_shared_gate, self.w_shared_gate_up = w_shared_gate, w_shared_gate_up
        self.w_shared_down = w_shared_down
        self.E, self.D = w_router.shape
        self.f = w_gate_up.shape[1] // 2
        self.f_s = 0 if w_shared_gate_up is None else w_shared_gate_up.shape[0] // 2
        self.K = K
        self.flags = (MOE_FLAG_DETERMINISTIC if deterministic else 0) | \
            (MOE_FLAG_BF16_WEIGHTS if bf16_weights else 0)
        self.score_mode = SCORES[score]
        self.select_bias = select_bias
        self.capacity_factor = float(capacity_factor)
        self.min_capacity = int(min_capacity)
        _check_rule(rule, self.E, w_router)
        self.rule = rule  # a route_rule(...) instead of score / select_bias / bf16_weights
        self._int8 = None
        self._ws = None
        self._ws_T = -1
        self._captured_ws = []
        self._copy_streams = None

    @classmethod
    def from_inputs(cls, inp, deterministic=False, **router):
        return cls(inp.w_router, inp.w_gate_up, inp.w_down, inp.cfg.K, inp.logit_bias,
                   inp.w_shared_gate, inp.w_shared_gate_up, inp.w_shared_down, deterministic,
                   **router)

    def workspace(self, T: int) -> torch.Tensor:
        if self._ws is None or self._ws_T < T:
            self._ws = alloc_workspace(T, self.D, self.E, self.K, self.f, self.f_s,
                                       self.w_router.device)
            self._ws_T = T
        return self._ws

    def _hold(self, ws, stream):
        """A graph that is being captured keeps the workspace's address, and work on another
        stream than the one the workspace was allocated on may outlast it: neither may find the
        memory in other hands once a larger batch has replaced the workspace."""
        if _capturing():
            if not any(w is ws for w in self._captured_ws):
                self._captured_ws.append(ws)
        else:
            ws.record_stream(stream)

    def params(self, x, topk_idx=None, topk_w=None, counts=None, events=None,
               residual=None) -> LayerParams:
        T = x.shape[0]
        ev = None if events is None else ctypes.cast(events, ctypes.c_void_p)
        return LayerParams(_p(x, BF16), _p(self.w_router, BF16), _p(self.logit_bias, F32),
                           _p(self.w_gate_up, BF16), _p(self.w_down, BF16),
                           _p(self.w_shared_gate, BF16), _p(self.w_shared_gate_up, BF16),
                           _p(self.w_shared_down, BF16), T, self.D, self.E, self.K, self.f,
                           self.f_s, self.flags, _p(topk_idx, I32), _p(topk_w, F32),
                           _p(counts, I32), ev, self.score_mode, _p(self.select_bias, F32),
                           _p(residual, BF16), self.capacity_factor, self.min_capacity)

    def __call__(self, x, out=None, topk_idx=None, topk_w=None, counts=None, stream=None,
                 step_events=None, residual=None):
        """y = layer(x) (+ residual h) on the device.  ``step_events``: an
        ``event_array(...)`` to time each kernel of the call."""
        T = x.shape[0]
        if x.shape[1] != self.D:
            raise MoEError(-1, "moe_layer_forward (x has the wrong width)")
        if self.rule is not None:
            _check_rule(self.rule, self.E, x)
        out = out if out is not None else torch.empty((T, self.D), dtype=torch.bfloat16,
                                                      device=x.device)
        ws = self.workspace(T)
        if stream is not None or _capturing():
            self._hold(ws, stream)
        prm = self.params(x, topk_idx, topk_w, counts, step_events, residual)
        if self.rule is None and self._int8 is None:
            rc = lib().moe_layer_forward(ctypes.byref(prm), _p(out, BF16), _p(ws, U8), ws.numel(),
                                         _stream(stream))
        else:
            rc = lib().moe_layer_forward_ex(ctypes.byref(prm), self.rule, self._int8,
                                            _p(out, BF16), _p(ws, U8), ws.numel(), _stream(stream))
        _check(rc, "moe_layer_forward")
        return out

    def plan(self, T: int):
        """(steps that launch kernels, kernels per call) for T tokens, from moe_layer_plan_ex:
        the step names of STEP_EVENT_NAMES whose interval holds work of their own."""
        x = torch.empty((0, self.D), dtype=BF16, device=self.w_router.device)
        prm = self.params(x)
        prm.T = T
        mask, n = ctypes.c_uint(0), ctypes.c_int(0)
        _check_rule(self.rule, self.E, x)
        _check(lib().moe_layer_plan_ex(ctypes.byref(prm), self.rule, ctypes.byref(mask), ctypes.byref(n)),
               "moe_layer_plan_ex")
        steps = [name for i, name in enumerate(STEP_EVENT_NAMES) if mask.value >> i & 1]
        return steps, n.value

    def forward_host(self, x_host, y_host, x_dev, y_dev, stream=None):
        """End to end from host memory: copy x (pinned host) in, run the layer, copy y
        out to pinned host memory; everything enqueued on one stream."""
        x_dev.copy_(x_host, non_blocking=True)
        self(x_dev, out=y_dev, stream=stream)
        y_host.copy_(y_dev, non_blocking=True)
        return y_host

    def forward_host_stream(self, x_hosts, y_hosts, x_devs, y_devs, stream=None):
        """End to end for a sequence of batches from host memory, each batch's copies
        overlapping the layer on its neighbours: batch i's x (pinned host) goes in on a copy
        stream while batch i-1 runs, its y comes back to pinned host memory on another copy
        stream while batch i+1 runs.  x_devs and y_devs hold two device buffers each (used
        in turn).  The layer runs on `stream` (default: the current stream), which at the end
        waits for the last copy out; returns y_hosts."""
        cur = torch.cuda.current_stream() if stream is None else stream
        if self._copy_streams is None:
            self._copy_streams = (torch.cuda.Stream(device=cur.device),
                                  torch.cuda.Stream(device=cur.device))
        h2d, d2h = self._copy_streams
        start = torch.cuda.Event()
        start.record(cur)
        h2d.wait_event(start)
        d2h.wait_event(start)
        ran, out = [], []
        for i, (xh, yh) in enumerate(zip(x_hosts, y_hosts)):
            b = i % 2
            with torch.cuda.stream(h2d):
                if i >= 2:
                    h2d.wait_event(ran[i - 2])  # the layer is done with x buffer b
                x_devs[b].copy_(xh, non_blocking=True)
                arrived = torch.cuda.Event()
                arrived.record(h2d)
            cur.wait_event(arrived)
            if i >= 2:
                cur.wait_event(out[i - 2])  # y buffer b has been copied out
            self(x_devs[b], out=y_devs[b], stream=cur)
            done = torch.cuda.Event()
            done.record(cur)
            ran.append(done)
            with torch.cuda.stream(d2h):
                d2h.wait_event(done)
                yh.copy_(y_devs[b], non_blocking=True)
                copied = torch.cuda.Event()
                copied.record(d2h)
            out.append(copied)
        if out:
            cur.wait_event(out[-1])
        return y_hosts

    def device_status(self, stream=None) -> int:
        return read_device_status(self._ws, stream) if self._ws is not None else 0


class Int8MoELayer(MoELayer):
    """One MoE layer whose experts (and shared expert) are 8-bit integers.

    Made from the bf16 weights of a MoELayer, which are quantised per output channel on
    construction and not kept; the router and the shared gate stay bf16.  Same options and
    calls as MoELayer, without step_events and plan()."""

    def __init__(self, w_router, w_gate_up, w_down, K, logit_bias=None, w_shared_gate=None,
                 w_shared_gate_up=None, w_shared_down=None, deterministic=False, **options):
        super().__init__(w_router, w_gate_up, w_down, K, logit_bias, w_shared_gate,
                         w_shared_gate_up, w_shared_down, deterministic, **options)
        self.quantized = [None if w is None else quantize_rows(w)
                          for w in (w_gate_up, w_down, w_shared_gate_up, w_shared_down)]
        self.w_gate_up = self.w_down = self.w_shared_gate_up = self.w_shared_down = None
        ptrs = []
        for qs in self.quantized:
            ptrs += [None, None] if qs is None else [_p(qs[0], I8), _p(qs[1], F32)]
        self._int8 = Int8Weights(*ptrs)

    def workspace(self, T: int) -> torch.Tensor:
        n = int(lib().moe_layer_ex_workspace_size(T, self.D, self.E, self.K, self.f, self.f_s,
                                                  self.flags, 1))
        if n == 0:
            raise MoEError(-2, "moe_layer_ex_workspace_size")
        if self._ws is None or self._ws.numel() < n:
            self._ws = torch.empty(n, dtype=U8, device=self.w_router.device)
            self._ws[:256].zero_()
        return self._ws

    def __call__(self, x, *args, **kw):
        with torch.cuda.device(x.device):  # (the launches go to the current device)
            return super().__call__(x, *args, **kw)

    def plan(self, T: int):
        raise MoEError(-2, "moe_layer_plan (a layer in 8-bit integers)")
