"""Routing by a rule and the 8-bit integer products in 64 bits, with the error that the CUDA
path may have (test helper)."""
from __future__ import annotations

import numpy as np
import torch

BF16_HALF = 2.0 ** -8   # a bf16 rounding, relative
F32_HALF = 2.0 ** -24   # an fp32 rounding, relative


def f64(t):
    return t.detach().double().cpu().numpy()


def route(logits, K, score="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renorm=True,
          scale=1.0):
    """(idx [T,K], w [T,K], allowed error of w) by the definition, token by token."""
    r = f64(logits)
    T, E = r.shape
    b = np.zeros(E) if bias is None else f64(bias)
    S = E // n_group
    idx = np.zeros((T, K), np.int64)
    w = np.zeros((T, K))
    tol = np.zeros((T, K))
    for t in range(T):
        row = np.where(np.isnan(r[t]), -np.inf, np.minimum(r[t], float(np.finfo(np.float32).max)))
        live = row > -np.inf
        s = np.zeros(E)
        spread = 0.0
        if score == "sigmoid":
            s[live] = np.exp(-np.logaddexp(0.0, -row[live]))
        elif live.any():
            m = row[live].max()
            s[live] = np.exp(row[live] - m)
            s[live] /= s[live].sum()
        with np.errstate(invalid="ignore"):
            key = np.where(live, s + b, -np.inf)
        key[~(key > -np.inf)] = -np.inf
        live &= key > -np.inf
        # equal scores of unequal logits (saturated in 64 bits too) keep the logits' order
        tie = row if bias is None else np.zeros(E)
        gscore = []
        for g in range(n_group):
            top = sorted(key[g * S:(g + 1) * S], reverse=True)[:group_top]
            top = [v for v in top if v > -np.inf]
            gscore.append(sum(top) if top else -np.inf)
        # (a group judged by its best score likewise: scores that underflow in 64 bits differ)
        gtie = [tie[g * S:(g + 1) * S].max() if group_top == 1 else 0.0 for g in range(n_group)]
        kept = sorted(range(n_group), key=lambda g: (-gscore[g], -gtie[g], g))[:topk_group]
        cand = [e for e in range(E) if e // S in kept]
        pick = sorted(cand, key=lambda e: (-key[e], -tie[e] if key[e] > -np.inf else 0.0, e))[:K]
        idx[t] = pick
        sel = np.where(live[pick], s[pick], 0.0)
        if score == "softmax" and live.any():
            spread = float(np.max(row[live].max() - row[pick][live[pick]], initial=0.0))
        on = live[pick]
        if renorm and on.any():  # from the scores' logarithms: they may underflow, the ratios do not
            ls = -np.logaddexp(0.0, -row[pick][on]) if score == "sigmoid" else row[pick][on]
            ratio = np.exp(ls - ls.max())
            sel[on] = ratio / ratio.sum()
        w[t] = sel * scale
        # expf 2 ulp and its rounded argument (spread * 2^-24), up to 21 additions in either sum,
        # divisions and the scale; renormalising counts the scores' error twice
        tol[t] = (4 * min(spread, 120.0) + 80) * F32_HALF * np.abs(w[t]) + 1e-37
    return idx, w, tol


def quantise(x):
    """(q, scale) of rows in 64 bits: q exact whole numbers."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(-1)
    bad = ~np.isfinite(top)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.rint(127.0 * x / np.where(top > 0, top, 1.0)[..., None])
    q[bad] = 0
    return q, np.where(bad, np.nan, top / 127.0)


def linear(xq, xs, wq, ws):
    """(y, allowed error): int32 sum exact, its fp32 conversion and two products, one bf16."""
    y = (xq @ wq.T) * xs[:, None] * ws[None, :]
    return y, np.abs(y) * (BF16_HALF + 4 * F32_HALF) + 1e-38


def _expert_rows(a, xs, gu, gus, dn, dns):
    """Rows a [n, D] (whole numbers) with scales xs through one expert: (v [n, D], the error
    that v may have in fp32 before the bf16 rounding)."""
    f = dn.shape[1]
    z = (a @ gu.T) * xs[:, None] * gus[None, :]
    g, u = z[:, :f], z[:, f:]
    with np.errstate(over="ignore"):
        h = g / (1.0 + np.exp(-g)) * u
    q, hs = quantise(h)
    # Relative error of h in fp32: g and u carry a conversion and two products (3 roundings),
    # which SiLU multiplies by up to 1 + |g|; exp and the division take (2 + |g|) 2^-22 and 2^-22.
    delta = (12 + 8 * np.abs(g).max(1)) * 2.0 ** -23
    # the quotient 127 h / amax has the errors of h and of amax; where it is this near to a tie, q
    # may be the other neighbour
    top = np.abs(h).max(1)
    quot = 127.0 * np.abs(h) / np.where(top > 0, top, 1.0)[:, None]
    near = np.abs(np.abs(quot - np.rint(quot)) - 0.5) < 128 * 2 * delta[:, None]
    v = (q @ dn.T) * hs[:, None] * dns[None, :]
    # flips by one step; the scale's own error; the fp32 sums of slices (4) and of scaled values
    err = (near.astype(np.float64) @ np.abs(dn).T) * hs[:, None] * dns[None, :]
    err += (np.abs(q) @ np.abs(dn).T) * hs[:, None] * dns[None, :] * (delta[:, None] + 12 * F32_HALF)
    return v, err


def experts(xq, xs, idx, w, gu, gus, dn, dns, keep=None, residual=None, shared=None):
    """(y, allowed error) of the routed experts for idx/w [T, K] (numpy, 64 bits); keep [T, K]:
    assignments that count; shared: (gate [T], gu, gus, dn, dns) of a shared expert."""
    T, K = idx.shape
    D = dn.shape[1]
    y, err, size = np.zeros((T, D)), np.zeros((T, D)), np.zeros((T, D))
    for e in range(gu.shape[0]):
        t, k = np.nonzero((idx == e) & (True if keep is None else keep))
        if len(t) == 0:
            continue
        v, dv = _expert_rows(xq[t], xs[t], gu[e], gus[e], dn[e], dns[e])
        np.add.at(y, t, v * w[t, k][:, None])
        np.add.at(err, t, dv * np.abs(w[t, k])[:, None])
        np.add.at(size, t, np.abs(v * w[t, k][:, None]))
        if T * K // gu.shape[0] >= 128:
            # many rows per expert: the weighted rows pass through 16-bit integers in blocks of
            # 32 columns, rint(v 32767 / top) with top = max |v|: half a step is top / 65534, and
            # the factor's error of 2^-21 on numbers up to 32767 adds 1/64 of a step
            top = np.abs(v * w[t, k][:, None]).reshape(len(t), D // 32, 32).max(2)
            np.add.at(err, t, np.repeat(top, 32, axis=1) * (0.5 + 1 / 64) / 32767)
    if shared is not None:
        gate, *weights = shared
        v, dv = _expert_rows(xq, xs, *weights)
        y += v * gate[:, None]
        # the gate's dot product and sigmoid in fp32
        err += (dv + 1e-5 * np.abs(v)) * gate[:, None]
        size += np.abs(v * gate[:, None])
    if residual is not None:
        y = y + residual
        size = size + np.abs(residual)
    err += size * (4 * K + 8) * F32_HALF
    return y, err + (np.abs(y) + err) * BF16_HALF + 1e-38


def assert_within(got, want, allow, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (got.shape, want.shape)
    nan = np.isnan(want)
    np.testing.assert_array_equal(np.isnan(got), nan, err_msg=what)
    over = np.abs(got - want)[~nan] - allow[~nan]
    assert over.size == 0 or over.max() <= 0, (
        f"{what}: {int((over > 0).sum())} of {over.size} values off by more than allowed, worst "
        f"excess {over.max():.3e} (largest value {np.abs(want[~nan]).max():.3e})")


def channels(rows, cols, gen):
    """Random 8-bit weights [rows, cols] with channel scales, on the CPU."""
    w = torch.randn(rows, cols, generator=gen) / cols ** 0.5
    s = w.abs().amax(1) / 127
    return torch.round(w / s[:, None]).to(torch.int8), s
