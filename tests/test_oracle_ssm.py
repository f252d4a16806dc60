"""The oracle of the convolution and the scan against what it has to agree with: hand-worked cases,
itself cut into pieces, central differences and float64 reverse-mode differentiation."""
import numpy as np
import pytest
import torch

import oracle as O

from _bounds import Err, U


def _scan_inputs(B, L, D, N, G, seed):
    r = np.random.default_rng(seed)
    return dict(u=r.standard_normal((B, L, D)), raw=r.standard_normal((B, L, D)) - 1,
                A=-np.exp(r.standard_normal((D, N)) * 0.5), Bm=r.standard_normal((B, L, G, N)),
                Cm=r.standard_normal((B, L, G, N)), skip=r.standard_normal(D), z=r.standard_normal((B, L, D)),
                dt_bias=r.standard_normal(D) * 0.3)


def test_conv_by_hand():
    x = np.array([[[1.0], [2.0], [3.0]]])
    w = np.array([[10.0, 1.0]])                       # p[t] = 10 x[t-1] + x[t]
    out, win = O.conv_causal(x, w, np.array([0.5]), silu=False)
    assert out[0, :, 0].tolist() == [1.5, 12.5, 23.5] and win[0, :, 0].tolist() == [3.0]
    out, win = O.conv_causal(x, w, None, silu=False, window=np.array([[[7.0]]]), lens=[1])
    assert out[0, :, 0].tolist() == [71.0, 0.0, 0.0] and win[0, 0, 0] == 1.0


def test_scan_by_hand():
    # dt = log(1 + e^raw) = 1 at raw = log(e - 1); A = log(1/2): the state halves at every token
    raw = np.full((1, 3, 1), np.log(np.e - 1))
    A = np.full((1, 8), np.log(0.5))
    Bm = np.zeros((1, 3, 1, 8))
    Cm = np.zeros((1, 3, 1, 8))
    Bm[..., 0], Cm[..., 0] = 2.0, 3.0
    u = np.array([[[1.0], [0.0], [4.0]]])
    out, end = O.ssm_scan(u, raw, A, Bm, Cm, skip=np.array([10.0]))
    # h = 2, 1, 0.5 + 8
    np.testing.assert_allclose(out[0, :, 0], [6 + 10, 3, 25.5 + 40])
    np.testing.assert_allclose(end[0, 0, 0], 8.5)


@pytest.mark.parametrize("cut", [0, 1, 5, 11])
def test_pieces_continue(cut):
    s = _scan_inputs(2, 11, 4, 8, 2, 1)
    seq = ("u", "raw", "Bm", "Cm", "z")
    full, end = O.ssm_scan(**s)
    a, h = O.ssm_scan(**{k: v[:, :cut] if k in seq else v for k, v in s.items()})
    b, h = O.ssm_scan(**{k: v[:, cut:] if k in seq else v for k, v in s.items()}, state=h)
    np.testing.assert_allclose(np.concatenate([a, b], 1), full, rtol=1e-12)
    np.testing.assert_allclose(h, end, rtol=1e-12)
    w = np.random.default_rng(2).standard_normal((4, 4))
    full, end = O.conv_causal(s["u"], w)
    a, win = O.conv_causal(s["u"][:, :cut], w)
    b, win = O.conv_causal(s["u"][:, cut:], w, window=win)
    np.testing.assert_allclose(np.concatenate([a, b], 1), full, rtol=1e-12)
    np.testing.assert_array_equal(win, end)


def _torch_scan(s, lens):
    """An own float64 forward: every output as an explicit sum over the earlier tokens."""
    B, L, D = s["u"].shape
    rep = D // s["Bm"].shape[2]
    dt = torch.nn.functional.softplus(s["raw"] + s["dt_bias"])
    S = torch.cumsum(dt, 1)
    Bm, Cm = (s[k].repeat_interleave(rep, 2) for k in ("Bm", "Cm"))
    decay = torch.exp((S[:, :, None] - S[:, None])[..., None] * s["A"])        # [B, t, s, D, N]
    y = torch.einsum("btdn,btsdn,bsdn,bsd->btsd", Cm, decay, Bm, dt * s["u"])
    keep = torch.tril(torch.ones(L, L, dtype=torch.float64))
    y = torch.einsum("btsd,ts->btd", y, keep) + s["skip"] * s["u"]
    out = y * torch.nn.functional.silu(s["z"])
    return torch.stack([torch.where((torch.arange(L) < n)[:, None], o, torch.zeros_like(o))
                        for o, n in zip(out, lens)])


@pytest.mark.parametrize("lens", [[9, 9], [9, 4], [1, 0]])
def test_scan_backward_against_autograd(lens):
    s = _scan_inputs(2, 9, 6, 8, 3, 3)
    g = np.random.default_rng(4).standard_normal(s["u"].shape)
    t = {k: torch.tensor(v, requires_grad=True) for k, v in s.items()}
    out = _torch_scan(t, lens)
    np.testing.assert_allclose(out.detach().numpy(), O.ssm_scan(**s, lens=lens)[0], rtol=1e-10, atol=1e-12)
    names = ("u", "raw", "A", "Bm", "Cm", "skip", "z", "dt_bias")
    want = torch.autograd.grad(out, [t[k] for k in names], torch.tensor(g))
    got = O.ssm_scan_backward(**s, dout=g, lens=lens)
    for k, w, n in zip(("du", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias"), want, names):
        np.testing.assert_allclose(got[k], w.numpy(), rtol=1e-9, atol=1e-11, err_msg=k)


def test_scan_backward_against_differences():
    s = _scan_inputs(1, 5, 2, 8, 1, 5)
    g = np.random.default_rng(6).standard_normal(s["u"].shape)
    got = O.ssm_scan_backward(**s, dout=g)
    r = np.random.default_rng(7)
    for k, name in zip(("u", "raw", "A", "Bm", "Cm", "skip", "z", "dt_bias"),
                       ("du", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias")):
        d = r.standard_normal(s[k].shape)
        h = 1e-5
        up, dn = (np.sum(g * O.ssm_scan(**{**s, k: s[k] + e * h * d})[0]) for e in (1, -1))
        np.testing.assert_allclose(np.sum(got[name] * d), (up - dn) / (2 * h), rtol=1e-6, atol=1e-8, err_msg=name)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [2, 4])
def test_conv_backward_against_autograd(K, silu):
    r = np.random.default_rng(8)
    x, w, b, g = (r.standard_normal(s) for s in ((2, 7, 3), (3, K), (3,), (2, 7, 3)))
    lens = [7, 2]
    t = [torch.tensor(a, requires_grad=True) for a in (x, w, b)]
    xt = torch.where(torch.tensor([[i < n for i in range(7)] for n in lens])[..., None], t[0], 0.0)
    p = torch.nn.functional.conv1d(torch.nn.functional.pad(xt.transpose(1, 2), (K - 1, 0)), t[1][:, None], t[2],
                                   groups=3).transpose(1, 2)
    out = torch.nn.functional.silu(p) if silu else p
    m = torch.tensor([[i < n for i in range(7)] for n in lens])[..., None].double()
    want = torch.autograd.grad(out, t, torch.tensor(g) * m)
    np.testing.assert_allclose((out * m).detach().numpy(), O.conv_causal(x, w, b, silu, lens=lens)[0], rtol=1e-12,
                               atol=1e-14)
    for a, wnt in zip(O.conv_causal_backward(x, w, g, b, silu, lens), want):
        np.testing.assert_allclose(a, wnt.numpy(), rtol=1e-11, atol=1e-13)


def test_bounds_hold_for_fp32_arithmetic():
    """A float32 run of the oracle's own steps stays within the bounds that the tests allow, and the
    bounds are small next to the values."""
    s = {k: v.astype(np.float32) for k, v in _scan_inputs(2, 40, 6, 16, 2, 9).items()}
    g = np.random.default_rng(10).standard_normal(s["u"].shape).astype(np.float32)
    e = O.ssm_scan_backward(**{k: Err(v) for k, v in s.items()}, dout=Err(g))
    with np.errstate(over="ignore"):
        f = O.ssm_scan_backward(**s, dout=g)
    for k in e:
        assert (np.abs(f[k] - e[k].v) <= e[k].e + U * np.abs(e[k].v)).all(), k
        assert np.median(e[k].e / np.abs(e[k].v)) < 1e-3, k


def test_page_rules_by_hand():
    pool = np.arange(6.0)[:, None]
    out, done = O.pages_copy(pool, pool, [0, 0, 9, 1, 5, 2], [3, 4, 5, 4, 5, 0], same=True)
    #   0->3, 0->4, out of range, 4 named before, 5 named before, 0 is read by the call
    assert done == [1, 1, 0, 0, 0, 0] and out[:, 0].tolist() == [0, 1, 2, 0, 0, 5]
    out, table, live, where = O.pages_compact(pool, [5, -1, 1, 5, 7, 4])
    assert live == 3 and where == [-1, 1, -1, -1, 0, 2] and table == [2, -1, 1, 2, -1, 0]
    assert out[:3, 0].tolist() == [4, 1, 5]
