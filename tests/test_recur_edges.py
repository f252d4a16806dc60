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
