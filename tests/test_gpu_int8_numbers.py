"""Channel scales that are no numbers, or of extreme size, in the experts' 8-bit products: every
batch size answers with the NaN, the infinities and the numbers of the definition."""
import numpy as np
import pytest
import torch

import int8_ref as ref

pytestmark = pytest.mark.gpu

# tokens, experts: a handful of rows; weights on M; one-CTA tiles; CTA pairs (128 rows an expert)
BATCHES = [(3, 8), (12, 8), (40, 4), (600, 4), (900, 4)]


class Case:
    def __init__(self, T, E, D=512, K=2, f=128):
        g = torch.Generator().manual_seed(T + E)
        self.x = torch.randn(T, D, generator=g).bfloat16()
        parts = [ref.channels(2 * f, D, g) + ref.channels(D, f, g) for _ in range(E)]
        self.gu, self.gus, self.dn, self.dns = (torch.stack(v) for v in zip(*parts))
        self.idx = torch.argsort(torch.rand(T, E, generator=g), dim=1)[:, :K].int().contiguous()
        self.w = torch.rand(T, K, generator=g) + 0.05
        self.E = E

    def run(self, moe, deterministic=False):
        idx, w = self.idx.cuda(), self.w.cuda()
        counts = torch.bincount(idx.reshape(-1), minlength=self.E).int()
        perm = moe.permute(idx, w, counts, self.E)
        xq, xs = moe.quantize_rows(self.x.cuda())
        return moe.experts_int8(xq, xs, w, perm, self.gu.cuda(), self.gus.cuda(), self.dn.cuda(),
                                self.dns.cuda(), deterministic=deterministic)

    def want(self, dns=None):
        xq, xs = ref.quantise(ref.f64(self.x))
        with np.errstate(invalid="ignore", over="ignore"):
            return ref.experts(xq, xs, self.idx.numpy(), ref.f64(self.w), ref.f64(self.gu),
                               ref.f64(self.gus), ref.f64(self.dn),
                               ref.f64(self.dns if dns is None else dns))


@pytest.mark.parametrize("T,E", BATCHES)
@pytest.mark.parametrize("deterministic", [False, True])
def test_channel_scales_that_are_no_numbers(moe, T, E, deterministic):
    """Columns that no bad scale reaches are as if the bad channels were zero; the others hold
    the NaN and the infinities of the definition."""
    c = Case(T, E)
    inf, nan = float("inf"), float("nan")
    good = c.dns.clone()
    for e, d, s in ((0, 0, nan), (1, 77, inf), (2, 128, -inf), (3, 511, nan), (0, 300, nan), (1, 301, inf)):
        good[e, d], c.dns[e, d] = 0.0, s
    c.dns[2, 192:224] = nan  # a whole block
    good[2, 192:224] = 0.0
    y = ref.f64(c.run(moe, deterministic))
    bad, _ = c.want()
    want, allow = c.want(good)
    finite = np.isfinite(bad)
    np.testing.assert_array_equal(np.isnan(y), np.isnan(bad))
    np.testing.assert_array_equal(y[np.isinf(bad)], bad[np.isinf(bad)])
    assert (~finite).any() and finite.any()
    ref.assert_within(np.where(finite, y, 0), np.where(finite, want, 0), allow)


def test_a_weight_row_that_holds_a_nan(moe):
    """Through quantize_rows, as a layer makes its weights."""
    c = Case(600, 4)
    w = torch.randn(4, 512, 128, generator=torch.Generator().manual_seed(5)).bfloat16()
    w[1, 70, 3], w[2, 400, 100] = float("nan"), float("inf")
    q, s = moe.quantize_rows(w.cuda())
    c.dn, c.dns = q.cpu(), s.cpu()
    nan = torch.isnan(c.run(moe)).cpu()
    want = torch.zeros(600, 512, dtype=torch.bool)
    want[(c.idx == 1).any(1), 70] = True
    want[(c.idx == 2).any(1), 400] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("T,E", BATCHES)
def test_channel_scales_of_extreme_size(moe, T, E):
    """Down products around 1e-35 and 1e38 that their routing weights bring back to ordinary sizes."""
    c = Case(T, E)
    c.dns[0] *= 1e-36
    c.dns[1] *= 2e36
    c.dns[2, 64:96] = 0.0
    c.w[c.idx == 0] *= 1e36
    c.w[c.idx == 1] *= 1e-36
    y = c.run(moe)
    assert torch.isfinite(y).all()
    ref.assert_within(y, *c.want())
