"""Numbers that carry a bound on the rounding error that fp32 arithmetic can leave in them.

``Err(v, e)``: value v (float64) and a bound e >= 0 on how far the device's fp32
value can be from it.  Every operation adds what it can add:

  * a sum, product or quotient: half a step of fp32, U = 2^-24, of the result
    (4 U for a quotient: the approximate division is good to 2^-22);
  * e^x: the exponent's error, 3 U |x| for the product with log2 e and its own
    rounding, 2^-22 of the result for the hardware's power of two, and 2^-126,
    below which results may be flushed to zero;
  * log(1 + x): 4 U of the result (1 ulp, and 1 for what surrounds it);
  * a sum over n terms in any order: (n - 1) U of the sum of the magnitudes.

Running the oracle's functions on such numbers gives, beside the value, the
tolerance of every output, with no run of the device in it.  A device that
joins chunks sums exponents where the oracle multiplies powers: each of
these can lose about as much again, hence the factor 2 of ``tolerance``.
"""
import numpy as np

U = 2.0 ** -24


class Err:
    __array_priority__ = 100
    __array_ufunc__ = None

    def __init__(self, v, e=None):
        self.v = np.asarray(v, dtype=np.float64)
        self.e = np.zeros_like(self.v) if e is None else np.broadcast_to(np.asarray(e, np.float64), self.v.shape).copy()

    @staticmethod
    def of(x):
        return x if isinstance(x, Err) else Err(x)

    @property
    def shape(self):
        return self.v.shape

    def zeros(self, shape):
        return Err(np.zeros(shape))

    def __getitem__(self, i):
        return Err(self.v[i], self.e[i])

    def __setitem__(self, i, x):
        x = Err.of(x)
        self.v[i], self.e[i] = x.v, x.e

    def reshape(self, *s):
        return Err(self.v.reshape(*s), self.e.reshape(*s))

    def __neg__(self):
        return Err(-self.v, self.e)

    def __abs__(self):
        return Err(np.abs(self.v), self.e)

    def __add__(self, o):
        o = Err.of(o)
        v = self.v + o.v
        return Err(v, self.e + o.e + U * np.abs(v))

    __radd__ = __add__

    def __sub__(self, o):
        return self + (-Err.of(o))

    def __rsub__(self, o):
        return Err.of(o) + (-self)

    def __mul__(self, o):
        o = Err.of(o)
        v = self.v * o.v
        return Err(v, np.abs(self.v) * o.e + np.abs(o.v) * self.e + self.e * o.e + U * np.abs(v))

    __rmul__ = __mul__

    def __rtruediv__(self, o):
        v = o / self.v
        return Err(v, np.abs(v) * (self.e / np.maximum(np.abs(self.v) - self.e, 1e-300) + 4 * U))

    def exp(self):
        v = np.exp(self.v)
        return Err(v, v * (np.expm1(self.e + 3 * U * np.abs(self.v)) + 4 * U) + 2.0 ** -126)

    def log1p(self):
        v = np.log1p(self.v)
        return Err(v, self.e / np.maximum(1 + self.v - self.e, 1e-300) + 4 * U * np.abs(v))

    def sum(self, axis):
        n = self.v.shape[axis]
        return Err(self.v.sum(axis), self.e.sum(axis) + (n - 1) * U * np.abs(self.v).sum(axis))


def tolerance(x, dtype):
    """Bound of an output of the storage type: twice the arithmetic's, and half a step of the type
    (and of its smallest numbers: 2^-133 is half a step of bf16's, fp32's are finer)."""
    half = 2.0 ** -8 if dtype == "bf16" else U
    return 2 * x.e + half * (np.abs(x.v) + 2 * x.e) + 2.0 ** -126


def assert_within(got, want, dtype, name=""):
    got = np.asarray(got, np.float64)
    assert got.shape == want.v.shape, (name, got.shape, want.v.shape)
    tol = tolerance(want, dtype)
    bad = ~(np.abs(got - want.v) <= tol)
    assert not bad.any(), (name, int(bad.sum()), got.size, float(np.nanmax(np.abs(got - want.v) / tol)),
                           np.argwhere(bad)[:5].tolist())
