"""The 8-bit integer products on the tiles that large batches take: dense CTA pairs, dense tiles
of 128 and 256 weight rows, and a shared expert wide and long enough for CTA pairs."""
import numpy as np
import pytest
import torch

import int8_ref as ref
from workloads import LayerConfig, make_inputs

pytestmark = pytest.mark.gpu

# (T, N, K) by the launcher's rules on 148 SMs: CTA pairs from 128 rows on where 256 x 256 tiles
# number 37 or more, otherwise the widest of 256, 128 and 64 weight rows whose tiles (of 128
# tokens) are more than half of the SMs
DENSE = [(513, 3336, 272),    # CTA pairs: one row, 8 columns past the last whole tile
         (769, 2560, 144),    # CTA pairs: whole columns, K shorter than two steps
         (2304, 1048, 16),    # CTA pairs: whole rows, 24 columns in the last tile
         (700, 2056, 272),    # 128 weight rows
         (127, 9736, 400),    # 128: one row short, 8 columns in the last tile
         (100, 19208, 64),    # 256 weight rows
         (16, 32000, 528)]    # 256: a handful of rows, whole columns


@pytest.mark.parametrize("T,N,K", DENSE)
def test_int8_matmul(moe, T, N, K):
    g = torch.Generator().manual_seed(T + N + K)
    xq = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int8)
    wq = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    xs, ws = torch.rand(T, generator=g) + 0.1, torch.rand(N, generator=g) * 1e-3
    buf = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = moe.int8_matmul(xq.cuda(), xs.cuda(), wq.cuda(), ws.cuda(), out=buf[:T])
    assert bool((buf[T:] == 7).all())
    ref.assert_within(y, *ref.linear(ref.f64(xq), ref.f64(xs), ref.f64(wq), ref.f64(ws)), f"{T} {N} {K}")


@pytest.mark.parametrize("T,N,K", DENSE)
def test_linear_is_quantize_then_matmul(moe, T, N, K):
    """Bit for bit; NaN and infinite tokens and channel scales stay in their rows and columns."""
    g = torch.Generator().manual_seed(T * N + K)
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    x[3, 7], x[T - 1, K - 1] = float("nan"), float("inf")
    wq, ws = (t.cuda() for t in ref.channels(N, K, g))
    ws[5], ws[N - 1] = float("nan"), float("nan")
    y = moe.int8_linear(x, wq, ws)
    xq, xs = moe.quantize_rows(x)
    z = moe.int8_matmul(xq, xs, wq, ws)
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(z))
    nan = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    nan[3], nan[T - 1], nan[:, 5], nan[:, N - 1] = True, True, True, True
    assert torch.equal(torch.isnan(y), nan) and torch.equal(torch.isnan(z), nan)
    xs[[3, T - 1]], ws[[5, N - 1]] = 0.0, 0.0
    want, allow = ref.linear(ref.f64(xq), ref.f64(xs), ref.f64(wq), ref.f64(ws))
    ref.assert_within(torch.where(nan, 0.0, y), want, allow)


# shared expert: gate_up and down in CTA pairs (6 row blocks x 8 and 7 tiles; D ends in half a
# tile), and gate_up in tiles of 128 weight rows (3 row blocks x 26)
@pytest.mark.parametrize("T,D,fs", [(1300, 1664, 1024), (300, 256, 1664)])
@pytest.mark.parametrize("deterministic", [False, True])
def test_layer_with_a_wide_shared_expert(moe, T, D, fs, deterministic):
    E, K, f = 4, 2, 128
    inp = make_inputs(LayerConfig("int8_tiles", T=T, D=D, E=E, K=K, f=f, f_s=fs, seed=T)).to("cuda")
    layer = moe.Int8MoELayer.from_inputs(inp, deterministic=deterministic)
    idx = torch.empty((T, K), dtype=torch.int32, device="cuda")
    w = torch.empty((T, K), device="cuda")
    h = torch.randn(T, D, device="cuda", generator=torch.Generator("cuda").manual_seed(T)).bfloat16()
    y = layer(inp.x, topk_idx=idx, topk_w=w, residual=h)
    assert layer.device_status() == 0
    weights, shared = [], [1 / (1 + np.exp(-ref.f64(inp.x) @ ref.f64(inp.w_shared_gate)))]
    for t in (inp.w_gate_up, inp.w_down):
        weights += ref.quantise(ref.f64(t))
    for t in (inp.w_shared_gate_up, inp.w_shared_down):
        shared += ref.quantise(ref.f64(t))
    xq, xs = ref.quantise(ref.f64(inp.x))
    want, allow = ref.experts(xq, xs, idx.cpu().numpy(), ref.f64(w), *weights, residual=ref.f64(h),
                              shared=shared)
    # the scales are fp32 roundings of the 64-bit ones: three of them in a row's factors
    ref.assert_within(y, want, allow + np.abs(want) * 8 * ref.F32_HALF + 1e-6 * np.abs(want - ref.f64(h)))
