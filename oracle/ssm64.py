"""The short causal convolution, the selective state space scan (with their
gradients) and the page calls in plain float64 NumPy -- the oracle.

TEST INFRASTRUCTURE, like favor64.py: token by token from the definitions, no
chunks, no fusion.  The numeric functions take NumPy arrays, or any array-like
that offers the same indexing and arithmetic (the tests run them on numbers that
carry a rounding-error bound), through the few helpers below.

    convolution  p[t,c] = bias[c] + sum_k w[c,k] x[t-K+1+k, c];  out = p or p sigmoid(p)
    scan         dt = log(1 + e^(raw + dt_bias)),  h_n <- e^(dt A_n) h_n + dt u B_n,
                 y = sum_n C_n h_n + skip u,  out = y z sigmoid(z)
"""
from __future__ import annotations

import numpy as np

__all__ = ["conv_causal", "conv_causal_backward", "ssm_scan", "ssm_scan_backward", "pages_copy", "pages_compact"]


def _exp(x):
    return x.exp() if hasattr(x, "exp") else np.exp(x)


def _log1p(x):
    return x.log1p() if hasattr(x, "log1p") else np.log1p(x)


def _sum(x, axis):
    return x.sum(axis)


def _zeros(like, shape):
    return like.zeros(shape) if hasattr(like, "zeros") else np.zeros(shape)


def _sigmoid(x):
    # both halves by e^-|x|, so that nothing overflows
    e = _exp(-abs(x))
    r = 1.0 / (1.0 + e)
    neg = _value(x) < 0
    return r * np.where(neg, 0.0, 1.0) + (e * r) * np.where(neg, 1.0, 0.0)


def _value(x):
    return x.v if hasattr(x, "v") else x


def _softplus(x):
    return x * (_value(x) > 0) + _log1p(_exp(-abs(x)))


def _row_lens(lens, B, L):
    return [L] * B if lens is None else [max(0, min(L, int(n))) for n in lens]


def conv_causal(x, w, bias=None, silu=True, window=None, lens=None):
    """x [B, L, D], w [D, K], window [B, K-1, D] -> (out, window behind each row's end); rows of out
    behind a row's end are zero."""
    B, L, D = x.shape
    K = w.shape[1]
    out = _zeros(x, (B, L, D))
    win = _zeros(x, (B, K - 1, D))
    for b, n in enumerate(_row_lens(lens, B, L)):
        past = [_zeros(x, (D,)) if window is None else window[b, k] for k in range(K - 1)]
        seq = past + [x[b, t] for t in range(n)]
        for t in range(n):
            p = _zeros(x, (D,)) if bias is None else 1.0 * bias
            for k in range(K):
                p = p + w[:, k] * seq[t + k]
            out[b, t] = p * _sigmoid(p) if silu else p
        for k in range(K - 1):
            win[b, k] = seq[n + k]
    return out, win


def conv_causal_backward(x, w, dout, bias=None, silu=True, lens=None):
    """(dx, dw, dbias) of conv_causal from an empty past."""
    B, L, D = x.shape
    K = w.shape[1]
    dx = _zeros(x, (B, L, D))
    dw, db = _zeros(x, (D, K)), _zeros(x, (D,))
    for b, n in enumerate(_row_lens(lens, B, L)):
        g = []
        for t in range(n):
            p = _zeros(x, (D,)) if bias is None else 1.0 * bias
            for k in range(K):
                if t - K + 1 + k >= 0:
                    p = p + w[:, k] * x[b, t - K + 1 + k]
            s = _sigmoid(p)
            g.append(dout[b, t] * (s * (1.0 + p * (1.0 - s))) if silu else 1.0 * dout[b, t])
        for t in range(n):
            acc = _zeros(x, (D,))
            for k in range(K):
                if t + K - 1 - k < n:
                    acc = acc + w[:, k] * g[t + K - 1 - k]
                if t - K + 1 + k >= 0:
                    dw[:, k] = dw[:, k] + g[t] * x[b, t - K + 1 + k]
            dx[b, t] = acc
            db = db + g[t]
    return dx, dw, db


def _groups(m, D):
    """B or C of one token [G, N] -> [D, N]."""
    return m[np.arange(D) // (D // m.shape[0])]


def ssm_scan(u, raw, A, Bm, Cm, skip=None, z=None, dt_bias=None, state=None, lens=None):
    """-> (out [B, L, D], states [B, D, N] behind each row's end)."""
    B, L, D = u.shape
    N = A.shape[1]
    out = _zeros(u, (B, L, D))
    end = _zeros(u, (B, D, N))
    for b, n in enumerate(_row_lens(lens, B, L)):
        h = _zeros(u, (D, N)) if state is None else state[b]
        for t in range(n):
            dt = _softplus(raw[b, t] + dt_bias if dt_bias is not None else 1.0 * raw[b, t])
            h = _exp(dt[:, None] * A) * h + (dt * u[b, t])[:, None] * _groups(Bm[b, t], D)
            y = _sum(h * _groups(Cm[b, t], D), 1)
            if skip is not None:
                y = y + skip * u[b, t]
            out[b, t] = y * (z[b, t] * _sigmoid(z[b, t])) if z is not None else y
        end[b] = h
    return out, end


def ssm_scan_backward(u, raw, A, Bm, Cm, dout, skip=None, z=None, dt_bias=None, lens=None):
    """Gradients of ssm_scan from an empty past, as a dict (None where the input is None)."""
    B, L, D = u.shape
    N, G = A.shape[1], Bm.shape[2]
    du, ddt, dz = (_zeros(u, (B, L, D)) for _ in range(3))
    dB, dC = _zeros(u, (B, L, G, N)), _zeros(u, (B, L, G, N))
    dA, dskip, dbias = _zeros(u, (D, N)), _zeros(u, (D,)), _zeros(u, (D,))
    for b, n in enumerate(_row_lens(lens, B, L)):
        h, hs, a, dts, raws = _zeros(u, (D, N)), [], [], [], []
        for t in range(n):
            r = raw[b, t] + dt_bias if dt_bias is not None else 1.0 * raw[b, t]
            dt = _softplus(r)
            e = _exp(dt[:, None] * A)
            hs.append(h)
            h = e * h + (dt * u[b, t])[:, None] * _groups(Bm[b, t], D)
            a.append(e)
            dts.append(dt)
            raws.append(r)
        hs.append(h)
        mu = _zeros(u, (D, N))                       # a[t+1] lambda[t+1]
        for t in reversed(range(n)):
            Bt, Ct = _groups(Bm[b, t], D), _groups(Cm[b, t], D)
            g = 1.0 * dout[b, t]
            if z is not None:
                s = _sigmoid(z[b, t])
                y = _sum(hs[t + 1] * Ct, 1)
                if skip is not None:
                    y = y + skip * u[b, t]
                dz[b, t] = dout[b, t] * y * (s * (1.0 + z[b, t] * (1.0 - s)))
                g = dout[b, t] * (z[b, t] * s)
            lam = g[:, None] * Ct + mu
            dC[b, t] = _sum((g[:, None] * hs[t + 1]).reshape(G, D // G, N), 1)
            dB[b, t] = _sum((lam * (dts[t] * u[b, t])[:, None]).reshape(G, D // G, N), 1)
            mu = a[t] * lam
            q = mu * hs[t]
            lb = _sum(lam * Bt, 1)
            du[b, t] = dts[t] * lb + (skip * g if skip is not None else 0.0 * g)
            d = (u[b, t] * lb + _sum(q * A, 1)) * _sigmoid(raws[t])
            ddt[b, t] = d
            dA = dA + dts[t][:, None] * q
            dskip = dskip + g * u[b, t]
            dbias = dbias + d
    return dict(du=du, ddt=ddt, dA=dA, dB=dB, dC=dC, dskip=dskip if skip is not None else None,
                dz=dz if z is not None else None, ddt_bias=dbias if dt_bias is not None else None)


def pages_copy(dst_pool, src_pool, src, dst, same):
    """(dst pool after the call, done) by the rules of favor_pages_copy; same: one pool."""
    out, done = dst_pool.copy(), []
    for i, (s, d) in enumerate(zip(src, dst)):
        ok = 0 <= s < len(src_pool) and 0 <= d < len(dst_pool) and d not in list(dst[:i])
        if same and s != d and d in list(src):
            ok = False
        if ok:
            out[d] = src_pool[s]
        done.append(int(ok))
    return out, done


def pages_compact(pool, table):
    """(pool, new table, live pages, page map) by the rules of favor_pages_compact."""
    P = len(pool)
    live = sorted({p for p in table if 0 <= p < P})
    U = len(live)
    free = [p for p in range(U) if p not in live]
    where = [-1] * P
    for p in live:
        where[p] = p if p < U else free.pop(0)
    out = pool.copy()
    for p in live:
        out[where[p]] = pool[p]
    return out, [where[p] if 0 <= p < P else -1 for p in table], U, where
