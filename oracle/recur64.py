"""The gated linear recurrence and the group normalisation (with their gradients) in plain float64
NumPy -- the oracle.

TEST INFRASTRUCTURE, like ssm64.py: token by token from the definitions; the numeric functions take NumPy
arrays, or array-likes with the same indexing and arithmetic that carry a rounding-error bound.  (a h rather than
h - c h, so that a bound on h's error shrinks with h: |a| e, not (1 + c) e, which grows past any use in a long row.)

    recurrence  s = sigmoid(r + r_bias),  a = e^(-rate s)  (a = s without a rate),  w = 1, 1 - a or
                sqrt(1 - a^2),  h <- a h + w sigmoid(i + i_bias) x,  out = h z sigmoid(z)
    group norm  n = (x - mean) / sqrt(var + eps) over a token's groups,  u = n weight + bias,
                out = act(u), or u act(z)
"""
from __future__ import annotations

import numpy as np

from .ssm64 import _row_lens, _sigmoid, _sum, _value, _zeros

__all__ = ["recurrence", "recurrence_backward", "group_norm", "group_norm_backward"]


def _expm1(x):
    return x.expm1() if hasattr(x, "expm1") else np.expm1(x)


def _sqrt(x):
    return x.sqrt() if hasattr(x, "sqrt") else np.sqrt(x)


def _positive(x):
    return np.where(_value(x) > 0, 1.0, 0.0)


def _gates(r, rate, r_bias, scale):
    """(s, 1 - s, c = 1 - a, w, 1 / w or 0) of a token's row of raw gates."""
    raw = r if r_bias is None else r + r_bias
    s, sn = _sigmoid(raw), _sigmoid(-raw)
    c = sn if rate is None else -_expm1(-(rate * s))
    if scale == "plain":
        return s, sn, c, 1.0, 0.0
    if scale == "mean":
        return s, sn, c, c, 0.0
    q = c * (2.0 - c)                                 # 1 - a^2; where it is not positive w is 0
    on = _positive(q)
    w = _sqrt(q * on)
    return s, sn, c, w, on * (1.0 / (w + (1.0 - on)))


def _input(x, i, i_bias):
    """(sigmoid(i + i_bias), 1 - that, the gated input)."""
    if i is None:
        return 1.0, 0.0, 1.0 * x
    raw = i if i_bias is None else i + i_bias
    si = _sigmoid(raw)
    return si, _sigmoid(-raw), si * x


def _row(t, b, k):
    return None if t is None else t[b, k]


def recurrence(x, r, i=None, rate=None, r_bias=None, i_bias=None, z=None, scale="unit", state=None, lens=None):
    """x, r, i, z [B, L, D], state [B, D] -> (out, state behind each row's end); rows of out behind a
    row's end are zero."""
    B, L, D = x.shape
    out, end = _zeros(x, (B, L, D)), _zeros(x, (B, D))
    for b, n in enumerate(_row_lens(lens, B, L)):
        h = _zeros(x, (D,)) if state is None else state[b]
        for t in range(n):
            _, _, c, w, _ = _gates(r[b, t], rate, r_bias, scale)
            _, _, v = _input(x[b, t], _row(i, b, t), i_bias)
            h = (1.0 - c) * h + w * v
            out[b, t] = h if z is None else h * (z[b, t] * _sigmoid(z[b, t]))
        end[b] = h
    return out, end


def recurrence_backward(x, r, dout, i=None, rate=None, r_bias=None, i_bias=None, z=None, scale="unit", lens=None):
    """Gradients of recurrence from an empty past, as a dict (None where the input is None)."""
    B, L, D = x.shape
    g = {k: None if t is None else _zeros(x, (B, L, D)) for k, t in (("dx", x), ("dr", r), ("di", i), ("dz", z))}
    terms = [] if rate is None else _zeros(x, (B * L, D))        # of drate
    for b, n in enumerate(_row_lens(lens, B, L)):
        hs = [_zeros(x, (D,))]
        for t in range(n):
            _, _, c, w, _ = _gates(r[b, t], rate, r_bias, scale)
            _, _, v = _input(x[b, t], _row(i, b, t), i_bias)
            hs.append((1.0 - c) * hs[-1] + w * v)
        mu = _zeros(x, (D,))                                      # a lambda of the token behind
        for t in reversed(range(n)):
            s, sn, c, w, rw = _gates(r[b, t], rate, r_bias, scale)
            si, sin, v = _input(x[b, t], _row(i, b, t), i_bias)
            a, up = 1.0 - c, dout[b, t]
            if z is not None:
                zs, zn = _sigmoid(z[b, t]), _sigmoid(-z[b, t])
                g["dz"][b, t] = up * hs[t + 1] * (zs * (1.0 + z[b, t] * zn))
                up = up * (z[b, t] * zs)
            lam = up + mu
            mu = a * lam
            g["dx"][b, t] = lam * w * si
            if i is not None:
                g["di"][b, t] = lam * w * v * sin
            e = hs[t]
            if scale == "mean":
                e = e - v
            elif scale == "unit":
                e = e - v * (a * rw)
            aq = a * (lam * e)
            if rate is None:
                g["dr"][b, t] = aq * sn
            else:
                g["dr"][b, t] = -(aq * (rate * s * sn))
                terms[b * L + t] = -(aq * s)
    total = lambda t: _sum(t.reshape(B * L, D), 0)
    g["drate"] = None if rate is None else _sum(terms, 0)
    g["dr_bias"] = None if r_bias is None else total(g["dr"])
    g["di_bias"] = None if i_bias is None else total(g["di"])
    return g


def _act(name, x):
    """(f(x), f'(x))."""
    if name == "none":
        return x, 1.0
    if name == "silu":
        s, sn = _sigmoid(x), _sigmoid(-x)
        return x * s, s * (1.0 + x * sn)
    c, k = np.sqrt(2 / np.pi), 0.044715
    y = (2 * c) * (x * (1.0 + k * (x * x)))
    s, sn = _sigmoid(y), _sigmoid(-y)
    return x * s, s + x * s * sn * ((2 * c) * (1.0 + (3 * k) * (x * x)))


def _normalise(x, G, centred, eps):
    """x [T, D] -> (n [T * G, C], 1 / sqrt(var + eps) [T * G, 1])."""
    T, D = x.shape
    C = D // G
    x = x.reshape(T * G, C)
    if centred:
        x = x - (_sum(x, 1) * (1.0 / C)).reshape(T * G, 1)
    rstd = (1.0 / _sqrt(_sum(x * x, 1) * (1.0 / C) + eps)).reshape(T * G, 1)
    return x * rstd, rstd


def group_norm(x, G, weight=None, bias=None, z=None, act="none", centred=True, eps=1e-5, lens=None):
    """x, z [B, L, D] -> out; rows behind a row's end are zero."""
    B, L, D = x.shape
    out = _zeros(x, (B, L, D))
    for b, n in enumerate(_row_lens(lens, B, L)):
        if n:
            u = _normalise(x[b, :n], G, centred, eps)[0].reshape(n, D)
            u = u if weight is None else u * weight
            u = u if bias is None else u + bias
            out[b, :n] = _act(act, u)[0] if z is None else u * _act(act, z[b, :n])[0]
    return out


def group_norm_backward(x, dout, G, weight=None, bias=None, z=None, act="none", centred=True, eps=1e-5, lens=None):
    """Gradients of group_norm, as a dict (None where the input is None)."""
    B, L, D = x.shape
    C = D // G
    dx, dz, dws, dbs = (_zeros(x, (B, L, D)) for _ in range(4))
    for b, n in enumerate(_row_lens(lens, B, L)):
        if not n:
            continue
        nm, rstd = _normalise(x[b, :n], G, centred, eps)
        flat, up = nm.reshape(n, D), dout[b, :n]
        u = flat if weight is None else flat * weight
        u = u if bias is None else u + bias
        if z is None:
            du = up * _act(act, u)[1]
        else:
            f, df = _act(act, z[b, :n])
            du = up * f
            dz[b, :n] = up * u * df
        dws[b, :n] = du * flat
        dbs[b, :n] = du
        dn = (du if weight is None else du * weight).reshape(n * G, C)
        t = dn - nm * (_sum(dn * nm, 1) * (1.0 / C)).reshape(n * G, 1)
        if centred:
            t = t - (_sum(dn, 1) * (1.0 / C)).reshape(n * G, 1)
        dx[b, :n] = (rstd * t).reshape(n, D)
    total = lambda t: _sum(t.reshape(B * L, D), 0)
    return dict(dx=dx, dweight=None if weight is None else total(dws), dbias=None if bias is None else total(dbs),
                dz=None if z is None else dz)
