"""GPU tests of the group normalisation where a block takes several tiles of tokens: the next token's rows on their
way, the places of a wide group's sums in turn, the parameters' sums over tokens."""
import numpy as np
import pytest
import torch

import oracle as O
import random_feature_gb300 as R

from _bounds import U, Err, assert_within
from _util import to_dev, to_host
from test_group_norm import EPS, dev, errs, inputs
from test_recur import _round, ints

pytestmark = pytest.mark.gpu


def silu(z):
    s = 1.0 / (1.0 + (-z).exp())
    return z * s


# 32 or 16 tokens a tile and up to 608 blocks: 4 and 8 tiles a block; then groups that take a block, a token at a time
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,D,G,heads", [
    (3, 25000, 64, 4, False), (3, 25000, 64, 4, True), (3, 700, 1024, 1, False), (3, 600, 2048, 2, True),
    (3, 280, 12000, 2, False),
])
def test_several_tiles(B, L, D, G, heads, dtype):
    lens = [L, L // 2 + 1, 0]
    s = inputs(B, L, D, dtype, 70)
    g = _round(np.random.default_rng(71).standard_normal((B, L, D)), dtype)
    kw = dict(G=G, eps=EPS, act="silu", lens=lens)
    with R.GroupNorm(D, G, dtype, B, L, act="silu") as f:
        d, li = dev(s, dtype), ints(lens)
        if heads:
            d["x"] = d["x"].view(B, L, G, D // G).transpose(1, 2).contiguous()
        assert_within(to_host(f.norm(**d, lens=li)), O.group_norm(**errs(s), **kw), dtype, "out")
        got = f.backward(**d, dout=to_dev(g, dtype), lens=li)
        if heads:
            got["dx"] = got["dx"].transpose(1, 2).reshape(B, L, D)
    want = O.group_norm_backward(**errs(s), dout=Err(g), **kw)
    assert_within(to_host(got["dx"]), want["dx"], dtype, "dx")
    assert_within(to_host(got["dz"]), want["dz"], dtype, "dz")
    # The parameters' sums, whose bound over any order of 37501 terms would let a tile be lost: a term passes through
    # its block's tiles (up to 8 here), its tile's tokens (32) and the blocks' sums (3 and 3 and 5 of 608), under 64.
    for k in ("dweight", "dbias"):
        v, e, m = np.zeros(D), np.zeros(D), np.zeros(D)
        for b, n in enumerate(lens):
            if n:
                t = Err(g[b, :n]) * silu(Err(s["z"][b, :n]))
                if k == "dweight":
                    t = t * O.group_norm(Err(s["x"][b:b + 1, :n]), G, eps=EPS)[0]
                v, e, m = v + t.v.sum(0), e + t.e.sum(0), m + np.abs(t.v).sum(0)
        assert np.abs(v - want[k].v).max() <= 1e-9 * m.max()
        assert (np.abs(to_host(got[k]) - v) <= 2 * (e + 64 * U * m) + U * np.abs(v)).all(), k
