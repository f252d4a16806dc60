"""GPU tests of the selective scan and the short causal convolution (prompts, single tokens,
gradients) against the float64 oracle, with tolerances from running error bounds (_bounds.py)."""
import numpy as np
import pytest
import torch

import oracle as O
import random_feature_gb300 as R

from _bounds import Err, assert_within
from _util import to_dev, to_host

pytestmark = pytest.mark.gpu

SEQ = ("u", "raw", "Bm", "Cm", "z")
PAR = ("A", "skip", "dt_bias")


def _round(a, dtype):
    """The values that the storage type holds."""
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.float32 if dtype == "f32" else torch.bfloat16) \
        .double().numpy()


def scan_inputs(B, L, D, N, G, dtype, seed):
    r = np.random.default_rng(seed)
    step = np.exp(r.uniform(np.log(1e-3), np.log(1e-1), D))
    s = dict(u=r.standard_normal((B, L, D)), raw=0.5 * r.standard_normal((B, L, D)),
             Bm=r.standard_normal((B, L, G, N)), Cm=r.standard_normal((B, L, G, N)), z=r.standard_normal((B, L, D)))
    s = {k: _round(v, dtype) for k, v in s.items()}
    f32 = lambda a: a.astype(np.float32).astype(np.float64)
    s["A"] = f32(-np.arange(1, N + 1) * np.exp(0.3 * r.standard_normal((D, N))))
    s["skip"] = f32(r.standard_normal(D))
    s["dt_bias"] = f32(step + np.log(-np.expm1(-step)))
    return s


def dev(s, dtype):
    return {k: to_dev(v, dtype if k in SEQ or k in ("dout", "x") else "f32") for k, v in s.items() if v is not None}


def call_scan(f, d, **kw):
    return f.scan(d["u"], d["raw"], d["A"], d["Bm"], d["Cm"], skip=d.get("skip"), z=d.get("z"),
                  dt_bias=d.get("dt_bias"), **kw)


def call_step(f, d, t, state, **kw):
    z = d["z"][:, t].contiguous() if "z" in d else None
    return f.scan_step(*(d[k][:, t].contiguous() if k in SEQ else d[k] for k in ("u", "raw", "A", "Bm", "Cm")), state,
                       skip=d.get("skip"), z=z, dt_bias=d.get("dt_bias"), **kw)


def errs(s):
    return {k: Err(v) for k, v in s.items() if v is not None}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# B, L, D, N, G, lens: one token, odd widths, ragged rows, several groups, every N; long rows are cut into chunks
SCANS = [
    (1, 1, 1, 8, 1, None),
    (2, 7, 8, 16, 1, [7, 0]),
    (3, 65, 33, 16, 1, [65, 1, 64]),
    (2, 300, 72, 16, 3, [300, 129]),
    (1, 257, 40, 32, 5, None),
    (2, 130, 24, 64, 1, [2, 130]),
    (1, 200, 130, 8, 2, None),
]


def _id(c):
    return "x".join(str(v) for v in c[:5]) + ("_ragged" if c[5] else "")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SCANS, ids=_id)
def test_scan(case, dtype):
    B, L, D, N, G, lens = case
    s = scan_inputs(B, L, D, N, G, dtype, 1)
    h0 = np.random.default_rng(2).standard_normal((B, D, N)).astype(np.float32)
    want, end = O.ssm_scan(**errs(s), state=Err(h0), lens=lens)
    with R.Ssm(D, N, G, 4, dtype, B, L) as f:
        state = torch.from_numpy(h0).cuda()
        out = call_scan(f, dev(s, dtype), state=state, lens=None if lens is None else ints(lens))
        assert_within(to_host(out), want, dtype, "out")
        assert_within(to_host(state), end, "f32", "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("absent", [("skip",), ("z",), ("dt_bias",), ("skip", "z", "dt_bias")], ids="-".join)
def test_scan_absent_inputs(absent, dtype):
    s = scan_inputs(2, 90, 48, 16, 1, dtype, 3)
    g = _round(np.random.default_rng(4).standard_normal((2, 90, 48)), dtype)
    for k in absent:
        s[k] = None
    want, _ = O.ssm_scan(**errs(s))
    grads = O.ssm_scan_backward(**errs(s), dout=Err(g))
    with R.Ssm(48, 16, 1, 4, dtype, 2, 90) as f:
        d = dev(s, dtype)
        assert_within(to_host(call_scan(f, d)), want, dtype)
        got = f.scan_backward(d["u"], d["raw"], d["A"], d["Bm"], d["Cm"], to_dev(g, dtype), skip=d.get("skip"),
                              z=d.get("z"), dt_bias=d.get("dt_bias"))
        for k, w in grads.items():
            assert (got[k] is None) == (w is None), k
            if w is not None:
                assert_within(to_host(got[k]), w, dtype if k in ("du", "ddt", "dB", "dC", "dz") else "f32", k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_long(dtype):
    """Few channels and a long row: many chunks, the last one ragged."""
    s = scan_inputs(1, 2501, 40, 8, 1, dtype, 5)
    want, end = O.ssm_scan(**errs(s))
    with R.Ssm(40, 8, 1, 4, dtype, 1, 2501) as f:
        state = f.new_state(1)
        out = call_scan(f, dev(s, dtype), state=state)
        assert_within(to_host(out), want, dtype, "out")
        assert_within(to_host(state), end, "f32", "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_edges_of_the_step(dtype):
    """Raw steps from far below to far above: dt from an exact zero (the state stands still) to ones
    whose decay underflows to an exact zero; gates z that saturate both ways."""
    s = scan_inputs(1, 96, 16, 16, 1, dtype, 6)
    s["raw"] = _round(np.resize([-120.0, -30.0, 0.0, 25.0, 90.0, -2.0, 300.0], (1, 96, 16)), dtype)
    s["dt_bias"] = None
    s["z"] = _round(np.resize([-200.0, -90.0, 0.0, 90.0, 1.0], (1, 96, 16)), dtype)
    want, end = O.ssm_scan(**errs(s))
    with R.Ssm(16, 16, 1, 4, dtype, 1, 96) as f:
        state = f.new_state(1)
        out = to_host(call_scan(f, dev(s, dtype), state=state))
        assert_within(out, want, dtype)
        assert_within(to_host(state), end, "f32")
        g = f.scan_backward(*(dev(s, dtype)[k] for k in ("u", "raw", "A", "Bm", "Cm")), to_dev(np.ones_like(s["u"]), dtype),
                            z=to_dev(s["z"], dtype))
        for k, w in O.ssm_scan_backward(**errs({**s, "skip": None}), dout=Err(np.ones_like(s["u"]))).items():
            if w is not None:
                assert_within(to_host(g[k]), w, dtype if k in ("du", "ddt", "dB", "dC", "dz") else "f32", k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_state_without_decay_stands_still(dtype):
    """Steps whose softplus underflows to zero, and rates of zero, leave a state as it is to the last bit,
    through a prompt in chunks and through single tokens."""
    B, L, D, N = 1, 3000, 48, 16
    s = scan_inputs(B, L, D, N, 1, dtype, 38)
    s["skip"] = s["z"] = s["dt_bias"] = None
    h0 = torch.from_numpy(np.random.default_rng(39).standard_normal((B, D, N)).astype(np.float32)).cuda()
    with R.Ssm(D, N, 1, 4, dtype, B, L) as f:
        for still in ("raw", "A"):
            d = dev(s, dtype)
            if still == "raw":
                d["raw"].fill_(-200.0)              # dt = 0: nothing comes in, nothing decays
            else:
                d["A"].zero_()                      # nothing decays; nothing comes in either
                d["u"].zero_()
            state = h0.clone()
            call_scan(f, d, state=state)
            assert torch.equal(state, h0)
            for t in range(3):
                call_step(f, d, t, state)
            assert torch.equal(state, h0)


def test_nan_behind_a_row_stays_there():
    """Nothing behind a row's end is read or written."""
    B, L, D, N = 3, 140, 24, 16
    lens = [140, 0, 37]
    s = scan_inputs(B, L, D, N, 1, "bf16", 7)
    g = _round(np.random.default_rng(8).standard_normal((B, L, D)), "bf16")
    d, dd = dev(s, "bf16"), to_dev(g, "bf16")
    x = to_dev(s["u"], "bf16")
    for k in SEQ:
        for b, n in enumerate(lens):
            d[k][b, n:] = float("nan")
    for b, n in enumerate(lens):
        dd[b, n:] = float("nan")
        x[b, n:] = float("nan")
    li = ints(lens)
    with R.Ssm(D, N, 1, 4, "bf16", B, L) as f:
        out = torch.full_like(d["u"], 7.0)
        state = f.new_state(B)
        call_scan(f, d, lens=li, state=state, out=out)
        want, end = O.ssm_scan(**errs(s), lens=lens)
        for b, n in enumerate(lens):
            assert (to_host(out)[b, n:] == 7).all()
            out[b, n:] = 0
        assert_within(to_host(out), want, "bf16")
        assert_within(to_host(state), end, "f32")
        got = f.scan_backward(d["u"], d["raw"], d["A"], d["Bm"], d["Cm"], dd, skip=d["skip"], z=d["z"],
                              dt_bias=d["dt_bias"], lens=li)
        for k, w in O.ssm_scan_backward(**errs(s), dout=Err(g), lens=lens).items():
            assert_within(to_host(got[k]), w, "bf16" if k in ("du", "ddt", "dB", "dC", "dz") else "f32", k)
        w = np.random.default_rng(9).standard_normal((D, 4)).astype(np.float32)
        win = f.new_window(B)
        o = f.conv(x, to_dev(w, "f32"), lens=li, window=win)
        want, wend = O.conv_causal(Err(s["u"]), Err(w), lens=lens)
        assert_within(to_host(o), want, "bf16")
        np.testing.assert_array_equal(to_host(win), wend.v)
        dx, dw, _ = f.conv_backward(x, to_dev(w, "f32"), dd, lens=li)
        wx, ww, _ = O.conv_causal_backward(Err(s["u"]), Err(w), Err(g), lens=lens)
        assert_within(to_host(dx), wx, "bf16")
        assert_within(to_host(dw), ww, "f32")


def test_gradients_are_written_whole():
    """Through the C names into buffers full of NaN: behind a row's end the gradients are zero."""
    B, L, D, N = 3, 70, 24, 16
    lens = [70, 0, 33]
    s = scan_inputs(B, L, D, N, 1, "f32", 29)
    d = dev(s, "f32")
    g = to_dev(np.random.default_rng(30).standard_normal((B, L, D)), "f32")
    w = to_dev(np.random.default_rng(31).standard_normal((D, 4)), "f32")
    nan = lambda t: torch.full_like(t, float("nan"))
    with R.Ssm(D, N, 1, 4, "f32", B, L) as f:
        li = ints(lens)
        want = f.scan_backward(*(d[k] for k in ("u", "raw", "A", "Bm", "Cm")), g, skip=d["skip"], z=d["z"],
                               dt_bias=d["dt_bias"], lens=li)
        got = {k: nan(v) for k, v in want.items()}
        R.favor_ssm_scan_backward(f.handle, d["u"], d["raw"], d["A"], d["Bm"], d["Cm"], d["skip"], d["z"], d["dt_bias"],
                                  li, g, *got.values(), B, L)
        dx, dw = nan(d["u"]), nan(w)
        R.favor_conv_causal_backward(f.handle, d["u"], w, None, 1, li, g, dx, dw, None, B, L)
    for k, v in got.items():
        assert torch.equal(v, want[k]), k
    for b, n in enumerate(lens):
        for t in (dx, *(got[k] for k in ("du", "ddt", "dB", "dC", "dz"))):
            assert (t[b, n:] == 0).all() and torch.isfinite(t[b, :n]).all()


def test_infinite_gates():
    """Gates of either infinity: z sigmoid(z) is infinite above and has no value below, as its parts say."""
    s = scan_inputs(1, 4, 8, 8, 1, "f32", 32)
    for dtype in ("f32", "bf16"):
        d = dev(s, dtype)
        d["z"][0, 1] = float("inf")
        d["z"][0, 2] = float("-inf")
        with R.Ssm(8, 8, 1, 4, dtype, 1, 4) as f:
            out = to_host(call_scan(f, d))
        assert np.isinf(out[0, 1]).all() and np.isnan(out[0, 2]).all() and np.isfinite(out[0, [0, 3]]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SCANS, ids=_id)
def test_scan_backward(case, dtype):
    B, L, D, N, G, lens = case
    s = scan_inputs(B, L, D, N, G, dtype, 10)
    g = _round(np.random.default_rng(11).standard_normal((B, L, D)), dtype)
    want = O.ssm_scan_backward(**errs(s), dout=Err(g), lens=lens)
    with R.Ssm(D, N, G, 4, dtype, B, L) as f:
        d = dev(s, dtype)
        run = lambda: f.scan_backward(d["u"], d["raw"], d["A"], d["Bm"], d["Cm"], to_dev(g, dtype), skip=d["skip"],
                                      z=d["z"], dt_bias=d["dt_bias"], lens=None if lens is None else ints(lens))
        got = run()
        for k, w in want.items():
            assert_within(to_host(got[k]), w, dtype if k in ("du", "ddt", "dB", "dC", "dz") else "f32", k)
        for k, v in run().items():      # fixed-order sums
            assert torch.equal(v, got[k]), k


def test_scan_gradients_against_differences():
    """Central differences of the device's own forward call, fp32.  The call's result carries errors
    of at most `tolerance`; they and the h^2 term bound the quotient's error."""
    B, L, D, N = 1, 40, 8, 8
    s = scan_inputs(B, L, D, N, 1, "f32", 12)
    g = _round(np.random.default_rng(13).standard_normal((B, L, D)), "f32")
    from _bounds import tolerance
    with R.Ssm(D, N, 1, 4, "f32", B, L) as f:
        d = dev(s, "f32")
        got = f.scan_backward(d["u"], d["raw"], d["A"], d["Bm"], d["Cm"], to_dev(g, "f32"), skip=d["skip"], z=d["z"],
                              dt_bias=d["dt_bias"])
        h = 2.0 ** -6
        for k, name in (("u", "du"), ("raw", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("skip", "dskip"),
                        ("z", "dz"), ("dt_bias", "ddt_bias")):
            r = _round(np.random.default_rng(14).choice([-1.0, 1.0], s[k].shape), "f32")
            diff, slack, exact = 0.0, 0.0, {}
            for e in (1, -1):
                m = {**s, k: _round(s[k] + e * h * r, "f32")}
                diff += e * np.sum(g * to_host(call_scan(f, dev(m, "f32"))))
                w = O.ssm_scan(**errs(m))[0]
                slack += np.sum(np.abs(g) * tolerance(w, "f32"))
                exact[e] = np.sum(g * w.v)
            # what the quotient's own curvature makes of it, from the oracle
            true = np.sum(O.ssm_scan_backward(**s, dout=g)[name] * r)
            curve = abs((exact[1] - exact[-1]) / (2 * h) - true)
            mine = np.sum(to_host(got[name]) * r)
            own = np.sum(tolerance(O.ssm_scan_backward(**errs(s), dout=Err(g))[name], "f32"))
            assert abs(mine - diff / (2 * h)) <= slack / (2 * h) + curve + own, k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,G", [(8, 1), (16, 1), (32, 3), (64, 1)])
def test_prompt_then_tokens(N, G, dtype):
    """A prompt in two calls, then single tokens, over pages of a larger pool: the outputs and the
    states of one scan over everything; the same for the convolution."""
    B, L, D, P = 3, 75, 36, 7
    s = scan_inputs(B, L, D, N, G, dtype, 15)
    want, end = O.ssm_scan(**errs(s))
    pages = [5, 0, 3]
    pi = ints(pages)
    w = np.random.default_rng(16).standard_normal((D, 4)).astype(np.float32)
    bias = np.random.default_rng(17).standard_normal(D).astype(np.float32)
    cwant, cend = O.conv_causal(Err(s["u"]), Err(w), Err(bias))
    with R.Ssm(D, N, G, 4, dtype, B, L) as f:
        d = dev(s, dtype)
        part = lambda a, b: {k: v[:, a:b].contiguous() if k in SEQ else v for k, v in d.items()}
        state = torch.full((P, D, N), 9.0, device="cuda")
        win = torch.full((P, 3, D), 9.0, device="cuda", dtype=d["u"].dtype)
        R.pages_clear(state, pi)
        R.pages_clear(win, pi)
        outs = [call_scan(f, part(0, 60), state=state, pages=pi), call_scan(f, part(60, 71), state=state, pages=pi)]
        outs += [call_step(f, d, t, state, pages=pi)[:, None] for t in range(71, L)]
        assert_within(to_host(torch.cat(outs, 1)), want, dtype)
        assert_within(to_host(state[pages]), end, "f32")
        wd, bd = to_dev(w, "f32"), to_dev(bias, "f32")
        couts = [f.conv(d["u"][:, a:b].contiguous(), wd, bd, window=win, pages=pi) for a, b in ((0, 60), (60, 61),
                                                                                                (61, 71))]
        couts += [f.conv_step(d["u"][:, t].contiguous(), wd, win, bd, pages=pi)[:, None] for t in range(71, L)]
        assert_within(to_host(torch.cat(couts, 1)), cwant, dtype)
        np.testing.assert_array_equal(to_host(win[pages]), cend.v)
        rest = [p for p in range(P) if p not in pages]
        assert (to_host(state[rest]) == 9).all() and (to_host(win[rest]) == 9).all()


def test_rows_that_take_no_part():
    """Pages outside the pool (padding) and a page named twice: the first row has it."""
    B, D, N, P = 6, 40, 16, 4
    pages = [2, -1, 2, 4, 0, 2 ** 31 - 1]
    live = [0, 4]
    s = scan_inputs(B, 70, D, N, 1, "f32", 18)
    d = dev(s, "f32")
    pi = ints(pages)
    w = to_dev(np.random.default_rng(19).standard_normal((D, 3)), "f32")
    with R.Ssm(D, N, 1, 3, "f32", B, 70) as f:
        for step in (False, True):
            state, win = torch.full((P, D, N), 3.0, device="cuda"), torch.full((P, 2, D), 3.0, device="cuda")
            keep = [1, 3]
            if step:
                tok = {k: v[:, 0] if k in SEQ else v for k, v in d.items()}
                out = torch.full((B, D), 5.0, device="cuda")
                call_step(f, d, 0, state, pages=pi, out=out)
                ref = f.new_state(2) + 3
                one = {k: v[live].contiguous() if k in SEQ else v for k, v in d.items()}
                want = call_step(f, one, 0, ref)
                x = d["u"][:, 0].contiguous()
                co = f.conv_step(x, w, win, pages=pi)
                cref = f.new_window(2) + 3
                cw = f.conv_step(x[live].contiguous(), w, cref)
            else:
                out = torch.full((B, 70, D), 5.0, device="cuda")
                call_scan(f, d, state=state, pages=pi, out=out)
                ref = f.new_state(2) + 3
                want = call_scan(f, {k: v[live].contiguous() if k in SEQ else v for k, v in d.items()}, state=ref)
                co = f.conv(d["u"], w, window=win, pages=pi)
                cref = f.new_window(2) + 3
                cw = f.conv(d["u"][live].contiguous(), w, window=cref)
            dead = [b for b in range(B) if b not in live]
            assert (out[dead] == 0).all() and (co[dead] == 0).all()
            np.testing.assert_allclose(to_host(out[live]), to_host(want), rtol=1e-5, atol=1e-5)
            np.testing.assert_allclose(to_host(state[[2, 0]]), to_host(ref), rtol=1e-5, atol=1e-5)
            assert torch.equal(co[live], cw) and torch.equal(win[[2, 0]], cref)
            assert (state[keep] == 3).all() and (win[keep] == 3).all()


# B, L, D, K, lens
CONVS = [(1, 1, 1, 2, None), (1, 41, 64, 3, None), (2, 33, 48, 2, [30, 33]), (2, 5, 8, 4, [5, 0]), (3, 67, 33, 3, [67, 1, 2]), (2, 200, 72, 4, [130, 200]),
         (1, 129, 1030, 4, None)]


@pytest.mark.parametrize("silu", [True, False], ids=["silu", "linear"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CONVS, ids=lambda c: "x".join(str(v) for v in c[:4]))
def test_conv(case, dtype, silu):
    B, L, D, K, lens = case
    r = np.random.default_rng(20)
    x, g, win = (_round(r.standard_normal(s), dtype) for s in ((B, L, D), (B, L, D), (B, K - 1, D)))
    w, b = r.standard_normal((D, K)).astype(np.float32), r.standard_normal(D).astype(np.float32)
    li = None if lens is None else ints(lens)
    with R.Ssm(D, 8, 1, K, dtype, B, L) as f:
        xd, gd, wd, bd, wind = to_dev(x, dtype), to_dev(g, dtype), to_dev(w, "f32"), to_dev(b, "f32"), to_dev(win, dtype)
        out = f.conv(xd, wd, bd, silu=silu, window=wind, lens=li)
        want, end = O.conv_causal(Err(x), Err(w), Err(b), silu, Err(win), lens)
        assert_within(to_host(out), want, dtype)
        np.testing.assert_array_equal(to_host(wind), end.v)
        for bias in (None, b):
            dx, dw, db = f.conv_backward(xd, wd, gd, None if bias is None else bd, silu=silu, lens=li)
            wx, ww, wb = O.conv_causal_backward(Err(x), Err(w), Err(g), None if bias is None else Err(b), silu, lens)
            assert_within(to_host(dx), wx, dtype, "dx")
            assert_within(to_host(dw), ww, "f32", "dw")
            assert (db is None) == (bias is None)
            if db is not None:
                assert_within(to_host(db), wb, "f32", "db")


def test_long_runs():
    """A convolution large enough for runs of 128 tokens, bf16, against float64 on the device."""
    B, L, D, K = 2, 4096, 8192, 4
    g = torch.Generator(device="cuda").manual_seed(33)
    x = torch.randn(B, L, D, device="cuda", generator=g).bfloat16()
    w, b = torch.randn(D, K, device="cuda", generator=g), torch.randn(D, device="cuda", generator=g)
    lens = [L, 3001]
    with R.Ssm(D, 8, 1, K, "bf16", B, L, training=False) as f:
        out = f.conv(x, w, b, lens=ints(lens))
    for r, n in enumerate(lens):
        xp = torch.cat([x.new_zeros(K - 1, D), x[r, :n]]).double()
        p, mag = b.double().expand(n, D).clone(), b.double().abs().expand(n, D).clone()
        for k in range(K):
            p += w[:, k].double() * xp[k:k + n]
            mag += (w[:, k].double() * xp[k:k + n]).abs()
        want = p * torch.sigmoid(p)
        # |silu'| <= 1.1; K + 1 fp32 operations on terms of size mag; the gate to 2^-19 and for |p| >= 16 to |p| 2^-23
        tol = want.abs() * (2.0 ** -8 + 2.0 ** -18 + p.abs() * 2.0 ** -22) + 1.1 * mag * (K + 1) * 2.0 ** -24 + 2.0 ** -120
        assert ((out[r, :n].double() - want).abs() <= tol).all()
        assert (out[r, n:] == 0).all()


@pytest.mark.parametrize("N", [8, 64])
def test_many_blocks(N):
    """Enough channels for every SM without chunks, and a width that no tile divides."""
    B, L, D = 3, 21, 18001 if N == 8 else 2201
    s = scan_inputs(B, L, D, N, 1, "f32", 34)
    want, end = O.ssm_scan(**errs(s))
    with R.Ssm(D, N, 1, 4, "f32", B, L, training=False) as f:
        n = 4 * torch.cuda.get_device_properties(0).multi_processor_count
        assert B * -(-D // (2048 // N)) > n / 3
        state = f.new_state(B)
        assert_within(to_host(call_scan(f, dev(s, "f32"), state=state)), want, "f32")
        assert_within(to_host(state), end, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_rows_alone(dtype):
    """A batch whose summaries take several chunks a block, against its rows alone, where they take
    one: the same operations in the same order, so the same bits (sums over the batch aside)."""
    B, L, D, N = 4, 2048, 1024, 64
    s = scan_inputs(B, 1, D, N, 1, "f32", 35)
    g = torch.Generator(device="cuda").manual_seed(36)
    rn = lambda *sh: torch.randn(*sh, device="cuda", generator=g).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    u, raw, z, do, Bm, Cm = rn(B, L, D), rn(B, L, D), rn(B, L, D), rn(B, L, D), rn(B, L, 1, N), rn(B, L, 1, N)
    A, skip, bias = (to_dev(s[k], "f32") for k in ("A", "skip", "dt_bias"))
    with R.Ssm(D, N, 1, 4, dtype, B, L) as f:
        whole = f.scan_backward(u, raw, A, Bm, Cm, do, skip=skip, z=z, dt_bias=bias)
        rows = [f.scan_backward(*(t[b:b + 1] for t in (u, raw)), A, *(t[b:b + 1] for t in (Bm, Cm, do)), skip=skip,
                                z=z[b:b + 1], dt_bias=bias) for b in range(B)]
    for k in ("du", "ddt", "dz", "dB", "dC"):
        assert torch.equal(whole[k], torch.cat([r[k] for r in rows])), k


def test_offsets_past_32_bits():
    """A row of more than 2^31 elements against its second half alone, continued from the state; a pool of
    more than 2^31 states, stepped and copied at its far end."""
    D, N, L = 2048, 16, 1100000
    g = torch.Generator(device="cuda").manual_seed(37)
    rn = lambda *sh: torch.randn(*sh, device="cuda", generator=g, dtype=torch.bfloat16)
    u, raw, Bm, Cm = rn(1, L, D), rn(1, L, D), rn(1, L, 1, N), rn(1, L, 1, N)
    A = -torch.arange(1, N + 1, device="cuda").float().expand(D, N).contiguous()
    w = torch.randn(D, 4, device="cuda", generator=g)
    half = 1050000
    assert half * D > 2 ** 31
    with R.Ssm(D, N, 1, 4, "bf16", 1, L, training=False) as f:
        state, st2 = f.new_state(1), f.new_state(1)
        out = f.scan(u, raw, A, Bm, Cm, state=state)
        part = lambda t, a, b: t[:, a:b].contiguous()
        f.scan(*(part(t, 0, half) for t in (u, raw)), A, *(part(t, 0, half) for t in (Bm, Cm)), state=st2)
        tail = f.scan(*(part(t, half, L) for t in (u, raw)), A, *(part(t, half, L) for t in (Bm, Cm)), state=st2)
        # the two cut their tokens into other chunks: sums in fp32 that differ in their last places, which can
        # turn a rounding to bf16, so by one step of it, 2^-7 of the value at most
        assert (out[:, half:].float() - tail.float()).abs().max() <= 2.0 ** -7 * tail.float().abs().max()
        torch.testing.assert_close(state, st2, rtol=1e-4, atol=1e-5)
        del out, tail, raw
        win, w2 = f.new_window(1), f.new_window(1)
        c = f.conv(u, w, window=win)
        f.conv(part(u, 0, half), w, window=w2)
        assert torch.equal(c[:, half:], f.conv(part(u, half, L), w, window=w2)) and torch.equal(win, w2)
        del c, u, Bm, Cm
        P = 70000
        assert (P - 1) * D * N > 2 ** 31
        pool = torch.empty(P, D, N, device="cuda")
        pool[P - 1] = state[0]
        x, dt, B1, C1 = rn(1, D), rn(1, D), rn(1, 1, N), rn(1, 1, N)
        y = f.scan_step(x, dt, A, B1, C1, pool, pages=ints([P - 1]))
        assert torch.equal(y, f.scan_step(x, dt, A, B1, C1, state)) and torch.equal(pool[P - 1], state[0])
        assert R.pages_copy(pool, pool, ints([P - 1]), ints([P - 2])).item() == 1
        assert torch.equal(pool[P - 2], state[0])
        R.pages_clear(pool, ints([P - 2]))
        assert (pool[P - 2] == 0).all() and torch.equal(pool[P - 1], state[0])
        assert R.pages_compact(pool, ints([P - 1]))[0].item() == 0 and torch.equal(pool[0], state[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned_tensors(dtype):
    """Tensors one element past a 16-byte boundary take the paths of narrow accesses: the same
    operations in the same order, so the same bits."""
    B, L, D, N = 2, 50, 64, 16
    s = scan_inputs(B, L, D, N, 1, dtype, 21)
    from _util import to_dev_unaligned
    d = dev(s, dtype)
    o = {k: to_dev_unaligned(v, dtype) if k in SEQ else d[k] for k, v in s.items()}
    g = np.random.default_rng(22).standard_normal((B, L, D))
    w = to_dev(np.random.default_rng(23).standard_normal((D, 4)), "f32")
    with R.Ssm(D, N, 1, 4, dtype, B, L) as f:
        st = [f.new_state(B) for _ in range(2)]
        assert torch.equal(call_scan(f, d, state=st[0]), call_scan(f, o, state=st[1])) and torch.equal(*st)
        grads = [f.scan_backward(*(t[k] for k in ("u", "raw", "A", "Bm", "Cm")), gd, skip=t["skip"], z=t["z"],
                                 dt_bias=t["dt_bias"])
                 for t, gd in ((d, to_dev(g, dtype)), (o, to_dev_unaligned(g, dtype)))]
        for k in grads[0]:
            assert torch.equal(grads[0][k], grads[1][k]), k
        assert torch.equal(f.conv(d["u"], w), f.conv(o["u"], w))
        for a, b in zip(f.conv_backward(d["u"], w, to_dev(g, dtype)), f.conv_backward(o["u"], w, to_dev_unaligned(g, dtype))):
            assert a is None or torch.equal(a, b)


def test_captured_and_on_another_stream():
    """A decoding step (convolution and scan) captured into a graph and replayed on a side stream, and
    a training step of both, give what eager calls give."""
    B, D, N, T = 5, 96, 16, 4
    s = scan_inputs(B, T, D, N, 1, "bf16", 24)
    d = dev(s, "bf16")
    w = to_dev(np.random.default_rng(25).standard_normal((D, 4)), "f32")
    g = to_dev(np.random.default_rng(26).standard_normal((B, T, D)), "bf16")
    with R.Ssm(D, N, 1, 4, "bf16", B, T) as f:
        def step(t, win, state):
            x = f.conv_step(t["u"], w, win)
            return f.scan_step(x, t["raw"], t["A"], t["Bm"], t["Cm"], state, skip=t["skip"], z=t["z"],
                               dt_bias=t["dt_bias"])
        tok = lambda i: {k: v[:, i].contiguous() if k in SEQ else v for k, v in d.items()}
        win, state = f.new_window(B), f.new_state(B)
        want = [step(tok(i), win, state).clone() for i in range(T)]
        wstate = state.clone()
        win.zero_(), state.zero_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        inp = tok(0)
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = step(inp, win, state)
            for i in range(T):
                for k, v in tok(i).items():
                    inp[k].copy_(v)
                graph.replay()
                assert torch.equal(out, want[i])
        torch.cuda.synchronize()
        assert torch.equal(state, wstate)

        def train():
            x = f.conv(d["u"], w)
            gr = f.scan_backward(x, d["raw"], d["A"], d["Bm"], d["Cm"], g, skip=d["skip"], z=d["z"],
                                 dt_bias=d["dt_bias"])
            return [call_scan(f, {**d, "u": x}), *gr.values(), *f.conv_backward(d["u"], w, gr["du"])[:2]]
        want = [t.clone() for t in train()]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                got = train()
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_block_as_used():
    """A sequence block end to end: convolution, scan, then the gradients back through both, against
    the oracle's; the intermediate is the device's, rounded to the storage type."""
    B, L, D, N = 2, 150, 64, 16
    s = scan_inputs(B, L, D, N, 1, "f32", 27)
    r = np.random.default_rng(28)
    x = _round(r.standard_normal((B, L, D)), "f32")
    g = _round(r.standard_normal((B, L, D)), "f32")
    w, bias = r.standard_normal((D, 4)).astype(np.float32), r.standard_normal(D).astype(np.float32)
    d = dev(s, "f32")
    with R.Ssm(D, N, 1, 4, "f32", B, L) as f:
        u = f.conv(to_dev(x, "f32"), to_dev(w, "f32"), to_dev(bias, "f32"))
        out = call_scan(f, {**d, "u": u})
        gr = f.scan_backward(u, d["raw"], d["A"], d["Bm"], d["Cm"], to_dev(g, "f32"), skip=d["skip"], z=d["z"],
                             dt_bias=d["dt_bias"])
        dx, dw, db = f.conv_backward(to_dev(x, "f32"), to_dev(w, "f32"), gr["du"], to_dev(bias, "f32"))
    e = errs(s)
    wu, _ = O.conv_causal(Err(x), Err(w), Err(bias))
    e["u"] = wu
    want, _ = O.ssm_scan(**e)
    assert_within(to_host(out), want, "f32")
    wg = O.ssm_scan_backward(**e, dout=Err(g))
    for k, v in wg.items():
        assert_within(to_host(gr[k]), v, "f32", k)
    for a, b in zip((dx, dw, db), O.conv_causal_backward(Err(x), Err(w), wg["du"], Err(bias))):
        assert_within(to_host(a), b, "f32")


def test_gate_over_its_range():
    """x sigmoid(x) of fp32 storage, relative to its value, from where it vanishes to where it is x.
    With U = 2^-24: the exponential's 4 U and 1 U for the factor that mends its argument, 1 U each for
    1 + e, its reciprocal and the product, so 8 U; below 2^-126 the reciprocal may be flushed to zero."""
    x = np.concatenate([np.linspace(-90, 90, 40000), np.random.default_rng(40).uniform(-3, 3, 25536)])
    x = x.astype(np.float32).astype(np.float64).reshape(1, 64, 1024)
    with R.Ssm(1024, 8, 1, 2, "f32", 1, 64, training=False) as f:
        w = torch.tensor([0.0, 1.0], device="cuda").expand(1024, 2).contiguous()    # p = x
        got = to_host(f.conv(to_dev(x, "f32"), w))
    want = x / (1 + np.exp(-x))
    tol = 2.0 ** -21 * np.abs(want) + np.abs(x) * 2.0 ** -126
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("step", [False, True], ids=["prompt", "token"])
def test_step_size_over_its_range(step):
    """log(1 + e^x) of fp32 storage relative to its value: one token from an empty past with u = B_0 = C_0
    = 1 and A = 0 gives it back.  U = 2^-24: the exponential's 4 U and 1 U for the factor that mends its
    argument, 1 U for 2 + e, 2 U for its reciprocal, 1 U for their product, 1 U for the series and what
    it leaves out, 0.5 U for its inner terms, 1 U for the last sum, so 12 U."""
    D, N = 4096, 8
    r = np.random.default_rng(41)
    x = np.concatenate([np.linspace(-87, 95, 2048), r.uniform(-8, 4, 1024), r.uniform(-87, -20, 1024)])
    x = x.astype(np.float32).astype(np.float64).reshape(1, 1, D)
    one = np.zeros((1, 1, 1, N))
    one[..., 0] = 1
    d = [to_dev(a, "f32") for a in (np.ones((1, 1, D)), x, np.zeros((D, N)), one, one)]
    with R.Ssm(D, N, 1, 2, "f32", 1, 1, training=False) as f:
        if step:
            got = f.scan_step(*(t[:, 0].contiguous() if i != 2 else t for i, t in enumerate(d)), f.new_state(1))
        else:
            got = f.scan(*d)
    want = np.logaddexp(0, x)
    tol = 12 * 2.0 ** -24 * want + 2.0 ** -126
    err = np.abs(to_host(got).reshape(x.shape) - want)
    assert (err <= tol).all(), (np.max(err / tol), x.flat[np.argmax(err / tol)])


def test_step_size_of_infinities_and_nan():
    """log(1 + e^x) at both infinities, at the type's lowest value, behind its last exponential and of a NaN."""
    x = [float("inf"), float("-inf"), float("nan"), -3.4028234663852886e38, 3.4028234663852886e38, -128.5, 200.0, -1e4]
    D, N = len(x), 8
    for dtype in ("f32", "bf16"):
        raw = torch.tensor(x, device="cuda").view(1, 1, D).to(torch.float32 if dtype == "f32" else torch.bfloat16)
        one = torch.zeros(1, 1, 1, N, device="cuda", dtype=raw.dtype)
        one[..., 0] = 1
        with R.Ssm(D, N, 1, 2, dtype, 1, 1, training=False) as f:
            got = f.scan(torch.ones_like(raw), raw, torch.zeros(D, N, device="cuda"), one, one)
        got, raw = to_host(got).ravel(), to_host(raw).ravel()
        # what the type holds: bf16 rounds fp32's largest numbers to infinities; an infinite step meets
        # the zeros of B, which leaves no value
        fin = raw < np.inf
        assert np.isnan(got[np.isnan(raw)]).all() and not np.isfinite(got[raw == np.inf]).any()
        np.testing.assert_array_equal(got[fin], np.maximum(raw, 0)[fin])


def test_convolution_sums_of_long_runs():
    """dw and dbias of equal terms whose running fp32 sum rounds the same way at every step.  Runs of R =
    500 tokens, B = 230 of them: with U = 2^-24 the four terms of a group cost 2.25 U of their sum, the
    groups of a run half a U each, so (R / 4 + 1) / 2; of the runs' sums 16 meet in four levels, one U each,
    the B / 128 of a warp cost (B / 128 + 1) / 2, and the eight warps meet in three levels."""
    B, L, D, K = 230, 500, 512, 4
    c = 1 + 128 * 2.0 ** -23
    x, g = torch.ones(B, L, D, device="cuda"), torch.full((B, L, D), c, device="cuda")
    w, b = torch.randn(D, K, device="cuda"), torch.zeros(D, device="cuda")
    with R.Ssm(D, 8, 1, K, "f32", B, L) as f:
        _, dw, db = f.conv_backward(x, w, g, b, silu=False)
    tol = (2.25 + (L / 4 + 1) / 2 + 4 + (B / 128 + 1) / 2 + 3) * 2.0 ** -24
    for k in range(K):
        want = B * (L - (K - 1 - k)) * c
        assert np.abs(to_host(dw[:, k]) / want - 1).max() <= tol
    assert np.abs(to_host(db) / (B * L * c) - 1).max() <= tol


def test_parameter_sums_of_many_chunks():
    """dskip of equal terms whose running fp32 sum rounds the same way at every step, over 16384 chunks of 32
    tokens.  With U = 2^-24 a chunk's sum costs (32 + 1) / 2 U of it; 16 chunks meet in four levels, one U
    each, the 16384 / 128 sums of a warp cost (128 + 1) / 2, and the eight warps meet in three levels."""
    B, L, D, N = 8, 65536, 8, 8
    c = 1 + 2557 * 2.0 ** -23
    u = torch.full((B, L, D), c, device="cuda")
    one, bc, A = torch.ones_like(u), torch.zeros(B, L, 1, N, device="cuda"), torch.zeros(D, N, device="cuda")
    with R.Ssm(D, N, 1, 4, "f32", B, L) as f:
        got = f.scan_backward(u, one, A, bc, bc, one, skip=torch.ones(D, device="cuda"))["dskip"]
    tol = (16.5 + 4 + (B * L / 32 / 128 + 1) / 2 + 3) * 2.0 ** -24
    assert np.abs(to_host(got) / (B * L * c) - 1).max() <= tol


def _conv64(x, w, b):
    """One row [n, D] in float64 on the device: (inputs with K-1 zeros before them, p, sum of the terms' magnitudes)."""
    K = w.shape[1]
    xp = torch.cat([x.new_zeros(K - 1, x.shape[1]), x]).double()
    p, mag = b.double().expand(x.shape).clone(), b.double().abs().expand(x.shape).clone()
    for k in range(K):
        p += w[:, k].double() * xp[k:k + len(x)]
        mag += (w[:, k].double() * xp[k:k + len(x)]).abs()
    return xp, p, mag


# on 152 SMs: runs of 504 tokens, one a row, in one wave of blocks; of 256, two a row, in two waves
@pytest.mark.parametrize("B,L,D", [(115, 500, 2048), (8, 500, 56320)])
def test_longest_runs(B, L, D):
    """bf16; the last row is short."""
    K, U = 4, 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(42)
    x = torch.randn(B, L, D, device="cuda", generator=g).bfloat16()
    w, b = torch.randn(D, K, device="cuda", generator=g), torch.randn(D, device="cuda", generator=g)
    lens = [L] * (B - 1) + [L - 3]
    with R.Ssm(D, 8, 1, K, "bf16", B, L, training=False) as f:
        out = f.conv(x, w, b, lens=ints(lens))
    for r in {0, B // 2, B - 1}:
        n = lens[r]
        _, p, mag = _conv64(x[r, :n], w, b)
        want = p * torch.sigmoid(p)
        # |silu'| <= 1.1; K + 1 fp32 operations on terms of size mag; the gate to 2^-18, and for |p| >= 16 to |p| 2^-22
        tol = want.abs() * (2.0 ** -8 + 2.0 ** -18 + p.abs() * 2.0 ** -22) + 1.1 * mag * (K + 1) * U + 2.0 ** -120
        assert ((out[r, :n].double() - want).abs() <= tol).all()
        assert (out[r, n:] == 0).all()


# runs of 500 tokens, one a row; of 252, two a row, in two waves of blocks
@pytest.mark.parametrize("B,L,D", [(230, 500, 512), (8, 500, 28160)])
def test_longest_runs_backward(B, L, D):
    """fp32.  With s = sigmoid(p) good to 8 U of its value, s (1 + p (1 - s)) is off by 20 U (1 + |p|) at most, and
    by silu'' <= 1/2 times p's own error; dx is K terms of it, dw and dbias sums of R / 4 + rows / 128 + 11 levels."""
    K, U = 4, 2.0 ** -24
    g = torch.Generator(device="cuda").manual_seed(43)
    x, do = (torch.randn(B, L, D, device="cuda", generator=g) for _ in range(2))
    w, b = torch.randn(D, K, device="cuda", generator=g), torch.randn(D, device="cuda", generator=g)
    lens = [L] * (B - 1) + [L - 3]
    with R.Ssm(D, 8, 1, K, "f32", B, L) as f:
        dx, dw, db = f.conv_backward(x, w, do, b, lens=ints(lens))
    want = torch.zeros(K + 1, D, device="cuda", dtype=torch.float64)
    tol = torch.zeros_like(want)
    levels = L / 4 + 2 * B / 128 + 11
    for r, n in enumerate(lens):
        xp, p, mag = _conv64(x[r, :n], w, b)
        s = torch.sigmoid(p)
        gr = do[r, :n].double() * (s * (1 + p * (1 - s)))
        eg = do[r, :n].double().abs() * (20 * U * (1 + p.abs()) + 0.5 * (K + 1) * U * mag) + U * gr.abs()
        d, ed = torch.zeros_like(p), torch.zeros_like(p)
        for k in range(K):
            at = K - 1 - k                          # dx[t] += w[k] g[t + at]
            t = w[:, k].double() * gr[at:]
            d[:n - at] += t
            ed[:n - at] += (K + 1) * U * t.abs() + w[:, k].double().abs() * eg[at:]
            term = gr * xp[k:k + n]
            want[k] += term.sum(0)
            tol[k] += levels * U * term.abs().sum(0) + (eg * xp[k:k + n].abs()).sum(0)
        want[K] += gr.sum(0)
        tol[K] += levels * U * gr.abs().sum(0) + eg.sum(0)
        assert ((dx[r, :n].double() - d).abs() <= ed + U * d.abs()).all(), r
        assert (dx[r, n:] == 0).all()
    got = torch.cat([dw.t(), db[None]]).double()
    assert ((got - want).abs() <= tol + U * want.abs()).all(), ((got - want).abs() / tol).max().item()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slow_decays(dtype):
    """Decays of 1e-5 to 1e-3 a token, whose errors add up over the whole row; through chunks, then through
    single tokens, and the gradients of the row's start."""
    B, L, D, N = 1, 3000, 16, 8
    s = scan_inputs(B, L, D, N, 1, dtype, 44)
    step = np.exp(np.random.default_rng(45).uniform(np.log(1e-5), np.log(1e-3), D))
    s["raw"] = _round(0.1 * s["raw"], dtype)
    s["dt_bias"] = np.log(np.expm1(step)).astype(np.float32).astype(np.float64)
    s["A"] = -np.ones((D, N))
    want, end = O.ssm_scan(**errs(s))
    T = 700
    part = {k: v[:, :T] if k in SEQ else v for k, v in s.items()}
    g = _round(np.random.default_rng(46).standard_normal((B, T, D)), dtype)
    grads = O.ssm_scan_backward(**errs(part), dout=Err(g))
    with R.Ssm(D, N, 1, 4, dtype, B, L) as f:
        d, state = dev(s, dtype), f.new_state(B)
        head = {k: v[:, :L - 20].contiguous() if k in SEQ else v for k, v in d.items()}
        outs = [call_scan(f, head, state=state)] + [call_step(f, d, t, state)[:, None] for t in range(L - 20, L)]
        assert_within(to_host(torch.cat(outs, 1)), want, dtype)
        assert_within(to_host(state), end, "f32")
        p = dev(part, dtype)
        got = f.scan_backward(p["u"], p["raw"], p["A"], p["Bm"], p["Cm"], to_dev(g, dtype), skip=p["skip"], z=p["z"],
                              dt_bias=p["dt_bias"])
        for k, w in grads.items():
            assert_within(to_host(got[k]), w, dtype if k in ("du", "ddt", "dB", "dC", "dz") else "f32", k)
