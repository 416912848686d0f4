"""Ways of calling the binding's functions, on the CPU as far as their own checks."""
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
import top_routing_grouped_03_b200 as moe
from top_routing_grouped_03_b200 import build as moe_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe_build.build()
    return moe.lib()


X = torch.zeros(4, 64, dtype=torch.bfloat16)
W, S = torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
NAMED = [(moe.route_logits, dict(logits=torch.zeros(4, 64), K=4)),
         (moe.quantize_rows, dict(x=X)),
         (moe.int8_matmul, dict(xq=W, x_scale=S, wq=W, w_scale=S)),
         (moe.int8_linear, dict(x=X, wq=W, w_scale=S)),
         (moe.experts_int8, dict(xq=W, x_scale=S, topk_w=S, perm={}, w_gate_up=W, gate_up_scale=S, w_down=W,
                                 down_scale=S))]


@pytest.mark.parametrize("call,kw", NAMED, ids=lambda v: getattr(v, "__name__", ""))
def test_every_argument_by_name(call, kw):
    """(Host tensors: refused as such, also with a stream, by the names the signature has.)"""
    for extra in ({}, dict(stream=None)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(**kw, **extra)
    first = next(iter(kw))
    rest = {k: v for k, v in kw.items() if k != first}
    with pytest.raises(TypeError, match=first):
        call(**rest)
    with pytest.raises(TypeError, match=first):
        call(kw[first], **kw)
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(kw[first], **rest)


WITHOUT_PRIVATE_NAMES = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import top_routing_grouped_03_b200 as moe
try:
    moe.quantize_rows(torch.zeros(4, 64, dtype=torch.bfloat16))
except ValueError as e:
    print("refused:", e)
assert moe._get_device is torch.cuda.current_device
torch.cuda.current_stream = lambda index: type("Stream", (), dict(cuda_stream=70 + index))
assert moe._raw_stream(3) == 73
"""


def test_a_torch_without_the_private_names_still_imports():
    """As a CPU build of torch is: the package imports, and its calls raise."""
    r = subprocess.run([sys.executable, "-c", WITHOUT_PRIVATE_NAMES], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "refused: expected a CUDA tensor" in r.stdout, r.stderr


def test_sizes_past_32_bits_are_refused():
    """Not cut to their low 32 bits on the way to the C ABI."""
    for bad in (2 ** 31, 2 ** 32 + 8, 2 ** 40):
        for sizes in ((bad,), (4, bad), (bad, 0), (-1, bad)):
            with pytest.raises(moe.MoEError) as e:
                moe._sizes("call", *sizes)
            assert e.value.code == -2
    moe._sizes("call", 0, 1, 2 ** 31 - 1)
    moe._sizes("call", -1, 4)  # (negative sizes are the library's to refuse)
    for kw in (dict(n_group=2 ** 32 + 2), dict(topk_group=2 ** 32 + 1), dict(group_top=2 ** 32 + 1)):
        with pytest.raises(moe.MoEError):
            moe.route_rule(64, 2, **kw)


@pytest.mark.gpu
def test_tensors_past_32_bit_rows_are_refused():
    rows = 2 ** 32 + 1
    before = moe.launch_count()
    logits = torch.empty((rows, 1), dtype=torch.bfloat16, device="cuda")  # 8 GiB, never written
    with pytest.raises(moe.MoEError):
        moe.route_logits(logits, 1)
    del logits
    w = torch.empty((2 ** 28 + 8, 16), dtype=torch.int8, device="cuda")  # 2^32 values, in rows of 16
    x, s = torch.zeros(1, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(1, device="cuda")
    with pytest.raises(moe.MoEError):
        moe.int8_linear(x, w, s.expand(2 ** 28 + 8).contiguous())  # (more rows than the library takes)
    assert moe.launch_count() == before
