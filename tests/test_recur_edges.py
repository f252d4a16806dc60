"""GPU tests of the gated linear recurrence at the edges of its parameters: decays of exactly 1 and next to it,
gates at their type's lowest value."""
import numpy as np
import pytest
import torch

import oracle as O
import random_feature_gb300 as R

from _bounds import Err, assert_within
from _util import to_dev, to_host
from test_recur import SEQ, _round, check_grads, dev, errs, inputs

pytestmark = pytest.mark.gpu

# rates of a warp's channels: nothing is ever lost (whole groups take the short series), that beside fast channels,
# and states that grow where the gate is open
RATES = {"keep": [-0.0], "beside": [-0.0, 0.5, 0.0, 2.0, -0.0, 0.125], "grow": [-1.0, -0.0, -0.25]}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", ["plain", "mean", "unit"])
@pytest.mark.parametrize("D", [8, 5])
@pytest.mark.parametrize("rates", RATES)
def test_decays_of_one(rates, D, scale, dtype):
    """A rate of -0 (what -log of a decay of 1 is), and one below 0 under a gate so closed that its sigmoid is 0 in
    fp32: the state stays.  27 tokens are groups of 4 and 2 tokens and a rest; then the same tokens one by one."""
    B, L = 2, 27
    s = inputs(B, L, D, dtype, 30)
    s["rate"] = np.resize(RATES[rates], D)
    s["r_bias"] = None
    if rates == "grow":
        s["r"][:, 1::2] = -120.0
    h0 = np.random.default_rng(31).standard_normal((B, D)).astype(np.float32)
    g = _round(np.random.default_rng(32).standard_normal((B, L, D)), dtype)
    want, end = O.recurrence(**errs(s), scale=scale, state=Err(h0))
    with R.Recurrence(D, dtype, B, L, scale) as f:
        d = dev(s, dtype)
        state = torch.from_numpy(h0).cuda()
        assert_within(to_host(f.scan(**d, state=state)), want, dtype, "out")
        assert_within(to_host(state), end, "f32", "state")
        state = torch.from_numpy(h0).cuda()
        outs = [f.step(**{k: v[:, t].contiguous() if k in SEQ else v for k, v in d.items()}, state=state)
                for t in range(L)]
        assert_within(to_host(torch.stack(outs, 1)), want, dtype, "steps")
        assert_within(to_host(state), end, "f32", "state behind the steps")
        check_grads(f.backward(**d, dout=to_dev(g, dtype)), O.recurrence_backward(**errs(s), dout=Err(g), scale=scale),
                    dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rates", [[1e-6, 1e-5, 1e-4, 1e-3], [1e-6, 0.5, 1e-4, 1e-5, 2.0, 1e-3, 3e-6, 1e-2]],
                         ids=["slow", "beside_fast"])
def test_equal_decays_in_long_runs(rates, dtype):
    """Open gates give a channel the same decay at every token.  Over runs of 1024 tokens (160 rows, so that a row is
    cut into 8) what rounding leaves must not add up: a decay of 1 - 17.5 steps of fp32 that is kept as 1 - 17 or 18
    steps would."""
    B, L, D = 160, 8192, len(rates)
    r = np.random.default_rng(33)
    x = _round(np.abs(r.standard_normal((B, L, D))), dtype)
    g = _round(np.abs(r.standard_normal((B, L, D))), dtype)
    rate = np.array(rates, np.float32).astype(np.float64)
    a = np.exp(-rate)
    hs, lam = np.zeros((L + 1, B, D)), np.zeros((L + 1, B, D))
    for t in range(L):
        hs[t + 1] = a * hs[t] + x[:, t]
    for t in reversed(range(L)):
        lam[t] = g[:, t] + a * lam[t + 1]
    drate = -np.sum(a * lam[:L] * hs[:L], (0, 1))
    # All terms are positive, and independent roundings, uniform within half a step (2^-24 of the value, deviation
    # 2^-24 / sqrt 3), come to sqrt(L / 3) 2^-24 = 3.1e-6 in L tokens: five of it.  drate has the states', the
    # gradients' and its own sum's.
    near = 5 * np.sqrt(L / 3) * 2.0 ** -24
    with R.Recurrence(D, dtype, B, L, "plain") as f:
        d = dict(x=to_dev(x, dtype), r=to_dev(np.full((B, L, D), 40.0), dtype), rate=to_dev(rate, "f32"))
        state = f.new_state(B)
        out = to_host(f.scan(**d, state=state))
        assert np.abs(to_host(state) / hs[L] - 1).max() <= near
        got = f.backward(**d, dout=to_dev(g, dtype))
        assert np.abs(to_host(got["drate"]) / drate - 1).max() <= 3 * near
        if dtype == "f32":
            assert np.abs(out / hs[1:].transpose(1, 0, 2) - 1).max() <= near
            assert np.abs(to_host(got["dx"]) / lam[:L].transpose(1, 0, 2) - 1).max() <= near


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 5, 300])
def test_states_that_are_not_finite(L, dtype):
    """An infinite or NaN state stays in its own channel and row; rows without tokens leave theirs alone."""
    B, D = 3, 12
    s = inputs(B, L, D, dtype, 34)
    h0 = np.random.default_rng(35).standard_normal((B, D)).astype(np.float32)
    bad = h0.copy()
    bad[0, 3], bad[0, 8], bad[1, 0], bad[2, 1] = np.inf, np.nan, -np.inf, np.inf
    lens = [L, L, 0]
    want = O.recurrence(**errs(s), state=Err(h0), lens=lens)[0]
    reached = np.zeros((B, D), bool)
    reached[0, [3, 8]] = reached[1, 0] = True
    with R.Recurrence(D, dtype, B, L) as f:
        d = dev(s, dtype)
        state = torch.from_numpy(bad).cuda()
        out = f.scan(**d, state=state, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        outs = [(to_host(out), to_host(state))]
        if L == 1:
            state = torch.from_numpy(bad).cuda()
            pages = torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda")
            out = f.step(**{k: v[:, 0].contiguous() if k in SEQ else v for k, v in d.items()}, state=state, pages=pages)
            outs.append((to_host(out[:, None]), to_host(state)))
        lost = np.broadcast_to(reached[:, None], (B, L, D))
        want = Err(np.where(lost, 0, want.v), want.e)
        for got, st in outs:
            assert not np.isfinite(got[lost]).any()
            assert_within(np.where(lost, 0, got), want, dtype)
            assert (np.isfinite(st) == (np.isfinite(bad) & ~reached)).all()
            assert np.array_equal(st[2], bad[2].astype(np.float64))
