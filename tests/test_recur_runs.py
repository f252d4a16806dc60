"""GPU tests of the gated linear recurrence in runs of a hundred tokens and in its branch of slow rates, against the
float64 oracle with running error bounds."""
import numpy as np
import pytest
import torch

import oracle as O
import random_feature_gb300 as R

from _bounds import U, Err, assert_within
from _util import to_dev, to_host
from test_recur import SEQ, VEC, _round, dev, inputs, ints

pytestmark = pytest.mark.gpu


def slow(s, D):
    """Rates of the short series (all of a warp's below 0.125), some of them 0."""
    s["rate"] = np.exp(np.random.default_rng(60).uniform(np.log(1e-3), np.log(0.11), D)).astype(np.float32) \
        .astype(np.float64)
    s["rate"][::9] = 0.0


def reference(s, g, h0, lens, scale):
    """(out, end, gradients) of the oracle, rows of one length side by side as channels: a channel of a row
    knows of no other."""
    B, L, D = s["x"].shape
    out, end = Err(np.zeros((B, L, D))), Err(np.zeros((B, D)))
    grads, drate = {k: Err(np.zeros((B, L, D))) for k in ("dx", "dr", "di", "dz")}, 0.0
    for n in sorted(set(lens)):
        rows = [b for b in range(B) if lens[b] == n]
        flat = lambda t: Err(t[rows, :n].transpose(1, 0, 2).reshape(1, n, -1))
        back = lambda t: t.reshape(n, len(rows), D)
        put = lambda to, t: [to.__setitem__((b, slice(0, n)), t[:, k]) for k, b in enumerate(rows)]
        if n == 0:
            end[rows] = Err(h0[rows].astype(np.float64))
            continue
        e = {k: flat(s[k]) for k in SEQ}
        e.update({k: None if s[k] is None else Err(np.tile(s[k], len(rows))) for k in VEC})
        o, h = O.recurrence(**e, scale=scale, state=Err(h0[rows].reshape(1, -1)))
        gr = O.recurrence_backward(**e, dout=flat(g), scale=scale)
        put(out, back(o))
        end[rows] = h.reshape(len(rows), D)
        for k in grads:
            put(grads[k], back(gr[k]))
        if s["rate"] is not None:
            drate = drate + gr["drate"].v.reshape(len(rows), D).sum(0)
    return out, end, grads, drate


def sums(s, grads, lens):
    """(value, bound) of the parameters' gradients.  A token's term passes through the sums of its group (3), of its
    run's groups (52 at most here), of 8 runs (3) and of the rows' chunks (300 / 128 + 7): under 80.  (The oracle's own
    bound, for any order, would let half of it be lost.)"""
    ok = np.arange(s["x"].shape[1])[None, :, None] < np.array(lens)[:, None, None]
    terms = {"dr_bias": grads["dr"], "di_bias": grads["di"]}
    if s["rate"] is not None:       # dr is its term times rate (1 - s), a product good to a few U
        k = np.where(s["rate"] > 0, s["rate"], 1.0) / (1.0 + np.exp(s["r"] + s["r_bias"])) * ok
        k = np.where(k > 0, 1.0 / np.where(k > 0, k, 1.0), 0.0) * (s["rate"] > 0)
        dr = grads["dr"]
        terms["drate"] = Err(dr.v * k, (dr.e + 4 * U * np.abs(dr.v)) * k)
    for name, t in terms.items():
        v, e, m = t.v.sum((0, 1)), t.e.sum((0, 1)), np.abs(t.v).sum((0, 1))
        yield name, v, 2 * (e + 80 * U * m) + U * np.abs(v)


def compare(B, L, D, lens, scale, rates, dtype, seed):
    s = inputs(B, L, D, dtype, seed, rate=rates != "none")
    if rates in ("slow", "lifted"):
        slow(s, D)
    if rates == "lifted":       # one channel in the warp that has to take the general form, and takes all with it
        s["rate"][5] = 0.2
    h0 = np.random.default_rng(seed + 1).standard_normal((B, D)).astype(np.float32)
    g = _round(np.random.default_rng(seed + 2).standard_normal((B, L, D)), dtype)
    want, end, grads, drate = reference(s, g, h0, lens, scale)
    with R.Recurrence(D, dtype, B, L, scale) as f:
        d, li = dev(s, dtype), ints(lens)
        state = torch.from_numpy(h0).cuda()
        assert_within(to_host(f.scan(**d, state=state, lens=li)), want, dtype, "out")
        assert_within(to_host(state), end, "f32", "state")
        got = f.backward(**d, dout=to_dev(g, dtype), lens=li)      # of an empty past, as the oracle's
    for k, w in grads.items():
        assert_within(to_host(got[k]), w, dtype, k)
    for k, v, tol in sums(s, grads, lens):
        if k == "drate":            # (a rate of 0 leaves dr none of it)
            on = s["rate"] > 0
            assert np.allclose(v[on], drate[on], rtol=1e-9, atol=1e-9 * np.abs(drate).max())
            tol = np.where(on, tol, np.inf)
        assert (np.abs(to_host(got[k]) - v) <= tol).all(), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rates", ["slow", "lifted"])
@pytest.mark.parametrize("scale", ["unit", "plain", "mean"])
def test_slow_rates(scale, rates, dtype):
    """Two slabs of channels, one of them in part; 18 chunks of runs of 8 tokens, and a rest."""
    compare(1, 1101, 136, [1101], scale, rates, dtype, 61)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D,scale,rates", [
    (100, 2403, 4, "unit", "slow"), (160, 803, 4, "mean", "none"), (160, 803, 3, "plain", "general"),
    (100, 803, 132, "unit", "general"),
])
def test_long_runs(B, L, D, scale, rates, dtype):
    """Rows cut into 3 chunks (or 1) of 8 runs of 104 tokens, which end inside a chunk, a run or a group, or before
    them."""
    compare(B, L, D, [L - 1, 0, 2 * L // 3 - 2] + [L] * (B - 3), scale, rates, dtype, 64)
