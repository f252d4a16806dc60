"""ctypes binding of the gated linear recurrence and of the group normalisation of the C ABI
(include/favor.h), in the manner of the scan's: argument marshalling and checks only.
"""
from __future__ import annotations

import ctypes

from .favor import DTYPE_CODES, _check, _made_on, _ptr, _stream, lib
from .ssm import Ssm, _at, _kind, _raw_stream

__all__ = [
    "FAVOR_RECUR_PLAIN", "FAVOR_RECUR_MEAN", "FAVOR_RECUR_UNIT", "FAVOR_ACT_NONE", "FAVOR_ACT_SILU",
    "FAVOR_ACT_GELU_TANH",
    "favor_recur_create", "favor_recur_destroy", "favor_recur_scan", "favor_recur_step", "favor_recur_backward",
    "favor_norm_create", "favor_norm_destroy", "favor_group_norm", "favor_group_norm_backward",
    "Recurrence", "GroupNorm",
]

FAVOR_RECUR_PLAIN, FAVOR_RECUR_MEAN, FAVOR_RECUR_UNIT = range(3)
SCALE_CODES = {"plain": FAVOR_RECUR_PLAIN, "mean": FAVOR_RECUR_MEAN, "unit": FAVOR_RECUR_UNIT}
FAVOR_ACT_NONE, FAVOR_ACT_SILU, FAVOR_ACT_GELU_TANH = range(3)
ACT_CODES = {"none": FAVOR_ACT_NONE, "silu": FAVOR_ACT_SILU, "gelu_tanh": FAVOR_ACT_GELU_TANH}


def _code(codes, value, name):
    """The code of a choice given by its name or its code."""
    if isinstance(value, str):
        if value not in codes:
            raise ValueError(f"{name}: expected one of {', '.join(codes)}, got {value!r}")
        return codes[value]
    return int(value)


def favor_recur_create(D, scale, dtype, max_B, max_L, training=True) -> int:
    """Create a handle for D channels.  Returns the handle (int)."""
    h = ctypes.c_void_p()
    st = lib().favor_recur_create(ctypes.byref(h), int(D), _code(SCALE_CODES, scale, "scale"),
                                  int(DTYPE_CODES.get(dtype, dtype)), int(max_B), int(max_L), 1 if training else 0)
    _check(st, "favor_recur_create")
    return h.value


def favor_recur_destroy(h) -> None:
    _check(lib().favor_recur_destroy(h), "favor_recur_destroy")


def favor_recur_scan(h, x, r, i, rate, r_bias, i_bias, z, state, pages, n_pages, lens, clear, out, B, L,
                     stream=None) -> None:
    _check(lib().favor_recur_scan(h, _ptr(x), _ptr(r), _ptr(i), _ptr(rate), _ptr(r_bias), _ptr(i_bias), _ptr(z),
                                  _ptr(state), _ptr(pages), int(n_pages), _ptr(lens), int(clear), _ptr(out), int(B),
                                  int(L), _stream(stream, x)), "favor_recur_scan")


def favor_recur_step(h, x, r, i, rate, r_bias, i_bias, z, state, pages, n_pages, out, B, stream=None) -> None:
    _check(lib().favor_recur_step(h, _ptr(x), _ptr(r), _ptr(i), _ptr(rate), _ptr(r_bias), _ptr(i_bias), _ptr(z),
                                  _ptr(state), _ptr(pages), int(n_pages), _ptr(out), int(B), _stream(stream, x)),
           "favor_recur_step")


def favor_recur_backward(h, x, r, i, rate, r_bias, i_bias, z, lens, dout, dx, dr, di, drate, dr_bias, di_bias, dz, B,
                         L, stream=None) -> None:
    _check(lib().favor_recur_backward(h, _ptr(x), _ptr(r), _ptr(i), _ptr(rate), _ptr(r_bias), _ptr(i_bias), _ptr(z),
                                      _ptr(lens), _ptr(dout), _ptr(dx), _ptr(dr), _ptr(di), _ptr(drate),
                                      _ptr(dr_bias), _ptr(di_bias), _ptr(dz), int(B), int(L), _stream(stream, x)),
           "favor_recur_backward")


def favor_norm_create(D, G, act, centred, eps, dtype, max_B, max_L, training=True) -> int:
    """Create a handle for D channels in G groups.  Returns the handle (int)."""
    h = ctypes.c_void_p()
    st = lib().favor_norm_create(ctypes.byref(h), int(D), int(G), _code(ACT_CODES, act, "act"), 1 if centred else 0,
                                 float(eps), int(DTYPE_CODES.get(dtype, dtype)), int(max_B), int(max_L),
                                 1 if training else 0)
    _check(st, "favor_norm_create")
    return h.value


def favor_norm_destroy(h) -> None:
    _check(lib().favor_norm_destroy(h), "favor_norm_destroy")


def favor_group_norm(h, x, heads, weight, bias, z, lens, clear, out, B, L, stream=None) -> None:
    _check(lib().favor_group_norm(h, _ptr(x), int(heads), _ptr(weight), _ptr(bias), _ptr(z), _ptr(lens), int(clear),
                                  _ptr(out), int(B), int(L), _stream(stream, x)), "favor_group_norm")


def favor_group_norm_backward(h, x, heads, weight, bias, z, lens, dout, dx, dweight, dbias, dz, B, L,
                              stream=None) -> None:
    _check(lib().favor_group_norm_backward(h, _ptr(x), int(heads), _ptr(weight), _ptr(bias), _ptr(z), _ptr(lens),
                                           _ptr(dout), _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(dz), int(B), int(L),
                                           _stream(stream, x)), "favor_group_norm_backward")


def _fits(t, want):
    """Whether t is None, or a contiguous tensor of that (shape, dtype, device)."""
    return t is None or (_kind(t) == want and t.is_contiguous())


class _Owner:
    """What the two objects share: one handle on one device, and the checks."""

    def _own(self, D, dtype, max_B, max_L, create, destroy):
        import torch
        self.D, self.dtype, self.max_B, self.max_L = D, dtype, max_B, max_L
        self._destroy = destroy
        self.handle = create()
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self._t = torch.float32 if DTYPE_CODES.get(dtype, dtype) == DTYPE_CODES["f32"] else torch.bfloat16
        self._f32, self._i32, self._lib = torch.float32, torch.int32, lib()
        self._vec = ((D,), self._f32, self.device)

    _check_all = Ssm._check_all

    def _new(self, x, shape, stream, out):
        """The output, of x's kind and that shape."""
        if out is None:
            import torch
            new = torch.empty_like if x.dim() < 4 else lambda x: x.new_empty(shape)
            return new(x) if stream is None else _made_on(stream, self.device, lambda: new(x))
        self._check_all(((out, (shape, self._t, self.device), "out"),))
        return out

    def _grads(self, stream, **inputs):
        """Empty gradients as the inputs are (None where one is None), by their names."""
        import torch
        new = torch.empty_like
        made = _made_on(stream, self.device, lambda: tuple(None if t is None else new(t) for t in inputs.values()))
        return dict(zip(("d" + k for k in inputs), made))

    def close(self):
        if self.handle:
            self._destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Recurrence(_Owner):
    """Owns one handle of the gated linear recurrence; checks shapes, dtypes and devices before calling
    the C ABI.  Batches are token-major: x, r, i, z [B, L, D]; a step call takes the same without L.
    ``scale`` is the input's weight: "plain", "mean" or "unit".  ``training=False`` leaves the
    gradients' workspace out.

    ``scan`` and ``backward`` use the handle's workspace: of one object, such calls (and replays of graphs
    that hold them) must not overlap on the device; use an object a stream.  ``step`` uses none.

    A call with ``stream`` makes its outputs in that stream's order; that the inputs are ready there, and
    that whoever reads the outputs on another stream waits for the call, is the caller's to arrange."""

    def __init__(self, D, dtype, max_B, max_L, scale="unit", training=True):
        self.handle = None
        self.scale = scale
        self._own(D, dtype, max_B, max_L, lambda: favor_recur_create(D, scale, dtype, max_B, max_L, training),
                  favor_recur_destroy)

    def new_state(self, P):
        """P empty states [P, D]."""
        import torch
        return torch.zeros((P, self.D), dtype=torch.float32, device=self.device)

    def _args(self, x, dims, r, i, rate, r_bias, i_bias, z, state=None, pages=None, lens=None):
        """Checks; (shape of x, number of pages)."""
        if x.dim() != dims:
            raise ValueError(f"x: expected {dims} dimensions, got {list(x.shape)}")
        shape = tuple(x.shape)
        P, pool = 0, None
        if state is not None:
            P = state.shape[0] if state.dim() else 0
            if P == 0:      # its address is NULL, which means that there is none
                raise ValueError(f"state: expected at least one page [{self.D}], got {list(state.shape)}")
            pool = ((P, self.D), self._f32, self.device)
        if i_bias is not None and i is None:
            raise ValueError("i_bias: given without i")
        seq, vec, rows = (shape[:-1] + (self.D,), self._t, self.device), self._vec, (shape[:1], self._i32, self.device)
        # (a decoding step's time is the host's: the names are put together only for a refusal)
        if _fits(x, seq) and _fits(r, seq) and _fits(i, seq) and _fits(z, seq) and _fits(rate, vec) \
                and _fits(r_bias, vec) and _fits(i_bias, vec) and _fits(state, pool) and _fits(pages, rows) \
                and _fits(lens, rows):
            return shape, P
        self._check_all(((x, seq, "x"), (r, seq, "r"), (i, seq, "i"), (z, seq, "z"), (rate, vec, "rate"),
                         (r_bias, vec, "r_bias"), (i_bias, vec, "i_bias"), (state, pool, "state"),
                         (pages, rows, "pages"), (lens, rows, "lens")))
        return shape, P

    def scan(self, x, r, i=None, rate=None, r_bias=None, i_bias=None, z=None, state=None, pages=None, lens=None,
             out=None, stream=None):
        """The recurrence over x [B, L, D] with the raw decay gate r and the raw input gate i; with state
        (pages [P, D]) it continues each row's past and leaves the state behind the row's last token."""
        shape, P = self._args(x, 3, r, i, rate, r_bias, i_bias, z, state, pages, lens)
        clear = 1 if out is None else 0     # a new output has zeros behind a row's end, a given one is left as it is
        out = self._new(x, shape, stream, out)
        _check(self._lib.favor_recur_scan(self.handle, x.data_ptr(), r.data_ptr(), _at(i), _at(rate), _at(r_bias),
                                          _at(i_bias), _at(z), _at(state), _at(pages), P, _at(lens), clear,
                                          out.data_ptr(), shape[0], shape[1], _raw_stream(stream, self._index)),
               "favor_recur_scan")
        return out

    def step(self, x, r, state, i=None, rate=None, r_bias=None, i_bias=None, z=None, pages=None, out=None,
             stream=None):
        """One token a row, x [B, D]; the rows' states move on."""
        shape, P = self._args(x, 2, r, i, rate, r_bias, i_bias, z, state, pages)
        out = self._new(x, shape, stream, out)
        _check(self._lib.favor_recur_step(self.handle, x.data_ptr(), r.data_ptr(), _at(i), _at(rate), _at(r_bias),
                                          _at(i_bias), _at(z), _at(state), _at(pages), P, out.data_ptr(), shape[0],
                                          _raw_stream(stream, self._index)), "favor_recur_step")
        return out

    def backward(self, x, r, dout, i=None, rate=None, r_bias=None, i_bias=None, z=None, lens=None, stream=None):
        """Gradients of scan(x, r, i, rate, r_bias, i_bias, z, lens=lens) for the upstream gradient dout, as
        a dict: dx, dr, di, drate, dr_bias, di_bias, dz (None where the input is None)."""
        shape, _ = self._args(x, 3, r, i, rate, r_bias, i_bias, z, lens=lens)
        self._check_all(((dout, _kind(x), "dout"),))
        g = self._grads(stream, x=x, r=r, i=i, rate=rate, r_bias=r_bias, i_bias=i_bias, z=z)
        _check(self._lib.favor_recur_backward(self.handle, x.data_ptr(), r.data_ptr(), _at(i), _at(rate), _at(r_bias),
                                              _at(i_bias), _at(z), _at(lens), dout.data_ptr(),
                                              *(_at(t) for t in g.values()), shape[0], shape[1],
                                              _raw_stream(stream, self._index)), "favor_recur_backward")
        return g


class GroupNorm(_Owner):
    """Owns one handle of the group normalisation over D channels in G groups, with the activation ``act``
    ("none", "silu" or "gelu_tanh"); ``centred=False`` leaves the mean in.  x is [B, L, D], single tokens
    [B, D], or [B, G, L, D / G] as the attention calls write it; the gate z and the output are [B, L, D] (or
    [B, D]).  ``training=False`` leaves the gradients' workspace out.

    ``backward`` uses the handle's workspace: of one object, such calls (and replays of graphs that hold
    them) must not overlap on the device.  ``norm`` uses none.  Streams as for ``Recurrence``."""

    def __init__(self, D, G, dtype, max_B, max_L, act="none", centred=True, eps=1e-5, training=True):
        self.handle = None
        self.G, self.act, self.centred, self.eps = G, act, centred, eps
        self._own(D, dtype, max_B, max_L,
                  lambda: favor_norm_create(D, G, act, centred, eps, dtype, max_B, max_L, training),
                  favor_norm_destroy)

    def _args(self, x, weight, bias, z, lens):
        """Checks; (shape of the output, whether x is laid out by heads, B, L)."""
        dims = x.dim()
        if dims == 4:
            B, L = x.shape[0], x.shape[2]
            shape, kind = (B, L, self.D), (B, self.G, L, self.D // self.G)
        elif dims == 2 or dims == 3:
            shape = kind = tuple(x.shape[:-1]) + (self.D,)
            B, L = shape[0], shape[1] if dims == 3 else 1
        else:
            raise ValueError(f"x: expected 2, 3 or 4 dimensions, got {list(x.shape)}")
        rows, vec = ((B,), self._i32, self.device), self._vec
        like_x, like_out = (kind, self._t, self.device), (shape, self._t, self.device)
        if not (_fits(x, like_x) and _fits(z, like_out) and _fits(weight, vec) and _fits(bias, vec)
                and _fits(lens, rows)):
            self._check_all(((x, like_x, "x"), (z, like_out, "z"), (weight, vec, "weight"), (bias, vec, "bias"),
                             (lens, rows, "lens")))
        return shape, 1 if dims == 4 else 0, B, L

    def norm(self, x, weight=None, bias=None, z=None, lens=None, out=None, stream=None):
        """act(n weight + bias), or (n weight + bias) act(z) with the gate z."""
        shape, heads, B, L = self._args(x, weight, bias, z, lens)
        clear = 1 if out is None else 0
        out = self._new(x, shape, stream, out)
        _check(self._lib.favor_group_norm(self.handle, x.data_ptr(), heads, _at(weight), _at(bias), _at(z), _at(lens),
                                          clear, out.data_ptr(), B, L, _raw_stream(stream, self._index)),
               "favor_group_norm")
        return out

    def backward(self, x, dout, weight=None, bias=None, z=None, lens=None, stream=None):
        """Gradients of norm(x, weight, bias, z, lens) for the upstream gradient dout, as a dict: dx, dweight,
        dbias, dz (None where the input is None)."""
        shape, heads, B, L = self._args(x, weight, bias, z, lens)
        self._check_all(((dout, (shape, self._t, self.device), "dout"),))
        g = self._grads(stream, x=x, weight=weight, bias=bias, z=z)
        _check(self._lib.favor_group_norm_backward(self.handle, x.data_ptr(), heads, _at(weight), _at(bias), _at(z),
                                                   _at(lens), dout.data_ptr(), *(_at(t) for t in g.values()), B, L,
                                                   _raw_stream(stream, self._index)), "favor_group_norm_backward")
        return g


def declare(L) -> None:
    """Argument types of the entry points above."""
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    L.favor_recur_create.argtypes = [ctypes.POINTER(vp), i, i, i, i, i, i]
    L.favor_recur_destroy.argtypes = [vp]
    L.favor_recur_scan.argtypes = [vp] * 10 + [i, vp, i, vp, i, i, vp]
    L.favor_recur_step.argtypes = [vp] * 10 + [i, vp, i, vp]
    L.favor_recur_backward.argtypes = [vp] * 17 + [i, i, vp]
    L.favor_norm_create.argtypes = [ctypes.POINTER(vp), i, i, i, i, f, i, i, i, i]
    L.favor_norm_destroy.argtypes = [vp]
    L.favor_group_norm.argtypes = [vp, vp, i, vp, vp, vp, vp, i, vp, i, i, vp]
    L.favor_group_norm_backward.argtypes = [vp, vp, i] + [vp] * 9 + [i, i, vp]
    for name in __all__:
        if name.startswith("favor_"):
            getattr(L, name).restype = i
