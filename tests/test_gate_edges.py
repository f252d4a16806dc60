"""GPU tests of gates far below and far above what a sigmoid tells from 0 and 1, down to the type's lowest value."""
import numpy as np
import pytest
import torch

import oracle as O
import random_feature_gb300 as R
import test_group_norm as N
import test_recur as S

from _bounds import Err, assert_within
from _util import to_dev, to_host

pytestmark = pytest.mark.gpu

LOWEST = {"f32": float(torch.finfo(torch.float32).min), "bf16": float(torch.finfo(torch.bfloat16).min)}
# A gate this far down is 0, and so is its derivative, to 1e-60: what the oracle is given for everything below
# (its own numbers leave float64 there), with tolerances that hold 2^-126 at least.
FLOOR = -200.0


def far(shape, dtype, seed):
    """Gates, one in two of them far down."""
    z = np.random.default_rng(seed).standard_normal(shape)
    z.reshape(-1)[::2] = np.resize([LOWEST[dtype], -1e30, -1e13, -1e15, -300.0, -1e20, -95.0], z.reshape(-1)[::2].size)
    return S._round(z, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_norm_gate(act, dtype):
    B, L, D, G = 2, 9, 64, 2
    s = N.inputs(B, L, D, dtype, 40)
    s["z"] = far((B, L, D), dtype, 41)
    g = S._round(np.random.default_rng(42).standard_normal((B, L, D)), dtype)
    e = N.errs({**s, "z": np.maximum(s["z"], FLOOR)})
    grads = O.group_norm_backward(dout=Err(g), G=G, act=act, eps=N.EPS, **e)
    with R.GroupNorm(D, G, dtype, B, L, act=act) as f:
        d = N.dev(s, dtype)
        assert_within(to_host(f.norm(**d)), O.group_norm(G=G, act=act, eps=N.EPS, **e), dtype)
        got = f.backward(**d, dout=to_dev(g, dtype))
        for k, w in grads.items():
            assert_within(to_host(got[k]), w, dtype if k in ("dx", "dz") else "f32", k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_norm_without_gate(act, dtype):
    """The activation of what is normalised, from biases that put it far down."""
    B, L, D, G = 2, 9, 64, 2
    s = N.inputs(B, L, D, dtype, 43, gate=False)
    s["bias"][::2] = np.resize([LOWEST[dtype], -1e13, -1e20, -300.0], D // 2).astype(np.float32)
    g = S._round(np.random.default_rng(44).standard_normal((B, L, D)), dtype)
    e = N.errs({**s, "bias": np.maximum(s["bias"], FLOOR)})
    grads = O.group_norm_backward(dout=Err(g), G=G, act=act, eps=N.EPS, **e)
    with R.GroupNorm(D, G, dtype, B, L, act=act) as f:
        d = N.dev(s, dtype)
        assert_within(to_host(f.norm(**d)), O.group_norm(G=G, act=act, eps=N.EPS, **e), dtype)
        got = f.backward(**d, dout=to_dev(g, dtype))
        for k in ("dx", "dweight", "dbias"):
            assert_within(to_host(got[k]), grads[k], dtype if k == "dx" else "f32", k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [24, 7])
def test_recurrence_gates(D, dtype):
    """The output's gate z, and the input's gate i."""
    B, L = 2, 21
    s = S.inputs(B, L, D, dtype, 45)
    for k, seed in (("z", 46), ("i", 47)):
        s[k] = far((B, L, D), dtype, seed)
    g = S._round(np.random.default_rng(48).standard_normal((B, L, D)), dtype)
    e = S.errs({**s, "z": np.maximum(s["z"], FLOOR), "i": np.maximum(s["i"], FLOOR)})
    with R.Recurrence(D, dtype, B, L) as f:
        d = S.dev(s, dtype)
        assert_within(to_host(f.scan(**d)), O.recurrence(**e)[0], dtype)
        S.check_grads(f.backward(**d, dout=to_dev(g, dtype)), O.recurrence_backward(**e, dout=Err(g)), dtype)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gates_far_up(act):
    """Above, the gate is z itself and its derivative 1: u dout and u z, rounded once (the fp32 arithmetic in front
    of it, a few steps of 2^-24, is inside the 2^-7 beside the rounding of 2^-8)."""
    B, L, D, G = 1, 4, 64, 2
    s = N.inputs(B, L, D, "bf16", 49)
    s["z"] = S._round(np.resize([1e13, 300.0, 1e25, -LOWEST["bf16"] / 64], (B, L, D)), "bf16")
    g = S._round(np.random.default_rng(50).standard_normal((B, L, D)), "bf16")
    with R.GroupNorm(D, G, "bf16", B, L, act=act) as f:
        d = N.dev(s, "bf16")
        u = O.group_norm(s["x"], G, s["weight"], s["bias"])
        got = f.backward(**d, dout=to_dev(g, "bf16"))
        assert np.allclose(to_host(f.norm(**d)), u * s["z"], rtol=2.0 ** -7, atol=0)
        assert np.allclose(to_host(got["dz"]), u * g, rtol=2.0 ** -7, atol=1e-6)
