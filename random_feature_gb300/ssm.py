"""ctypes binding of the selective scan, the short causal convolution and the state
pages of the C ABI (include/favor.h).

Like the attention binding: argument marshalling and checks only, the functions
keep the C names, the stream defaults to torch's current stream on the tensor's
device, and nothing falls back to anything when the library is missing.
"""
from __future__ import annotations

import ctypes

from .favor import DTYPE_CODES, _check, _ptr, _stream, lib

__all__ = [
    "favor_ssm_create", "favor_ssm_destroy", "favor_conv_causal", "favor_conv_causal_step",
    "favor_conv_causal_backward", "favor_ssm_scan", "favor_ssm_scan_step", "favor_ssm_scan_backward",
    "favor_pages_copy", "favor_pages_clear", "favor_pages_compact", "favor_pages_move",
    "Ssm", "pages_copy", "pages_clear", "pages_compact",
]


def favor_ssm_create(D, N, G, K, dtype, max_B, max_L, training=True) -> int:
    """Create a handle for D channels, N states, G groups and K taps.  Returns the handle (int)."""
    h = ctypes.c_void_p()
    st = lib().favor_ssm_create(ctypes.byref(h), int(D), int(N), int(G), int(K), int(DTYPE_CODES.get(dtype, dtype)),
                                int(max_B), int(max_L), 1 if training else 0)
    _check(st, "favor_ssm_create")
    return h.value


def favor_ssm_destroy(h) -> None:
    _check(lib().favor_ssm_destroy(h), "favor_ssm_destroy")


def favor_conv_causal(h, x, weight, bias, silu, window, pages, n_pages, lens, out, B, L, stream=None) -> None:
    _check(lib().favor_conv_causal(h, _ptr(x), _ptr(weight), _ptr(bias), int(silu), _ptr(window), _ptr(pages),
                                   int(n_pages), _ptr(lens), _ptr(out), int(B), int(L), _stream(stream, x)),
           "favor_conv_causal")


def favor_conv_causal_step(h, x, weight, bias, silu, window, pages, n_pages, out, B, stream=None) -> None:
    _check(lib().favor_conv_causal_step(h, _ptr(x), _ptr(weight), _ptr(bias), int(silu), _ptr(window), _ptr(pages),
                                        int(n_pages), _ptr(out), int(B), _stream(stream, x)),
           "favor_conv_causal_step")


def favor_conv_causal_backward(h, x, weight, bias, silu, lens, dout, dx, dweight, dbias, B, L, stream=None) -> None:
    _check(lib().favor_conv_causal_backward(h, _ptr(x), _ptr(weight), _ptr(bias), int(silu), _ptr(lens), _ptr(dout),
                                            _ptr(dx), _ptr(dweight), _ptr(dbias), int(B), int(L),
                                            _stream(stream, x)), "favor_conv_causal_backward")


def favor_ssm_scan(h, u, dt, A, Bm, Cm, skip, z, dt_bias, state, pages, n_pages, lens, out, B, L,
                   stream=None) -> None:
    _check(lib().favor_ssm_scan(h, _ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(skip), _ptr(z),
                                _ptr(dt_bias), _ptr(state), _ptr(pages), int(n_pages), _ptr(lens), _ptr(out), int(B),
                                int(L), _stream(stream, u)), "favor_ssm_scan")


def favor_ssm_scan_step(h, u, dt, A, Bm, Cm, skip, z, dt_bias, state, pages, n_pages, out, B, stream=None) -> None:
    _check(lib().favor_ssm_scan_step(h, _ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(skip), _ptr(z),
                                     _ptr(dt_bias), _ptr(state), _ptr(pages), int(n_pages), _ptr(out), int(B),
                                     _stream(stream, u)), "favor_ssm_scan_step")


def favor_ssm_scan_backward(h, u, dt, A, Bm, Cm, skip, z, dt_bias, lens, dout, du, ddt, dA, dB, dC, dskip, dz,
                            ddt_bias, B, L, stream=None) -> None:
    _check(lib().favor_ssm_scan_backward(h, _ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(skip), _ptr(z),
                                         _ptr(dt_bias), _ptr(lens), _ptr(dout), _ptr(du), _ptr(ddt), _ptr(dA),
                                         _ptr(dB), _ptr(dC), _ptr(dskip), _ptr(dz), _ptr(ddt_bias), int(B), int(L),
                                         _stream(stream, u)), "favor_ssm_scan_backward")


def favor_pages_copy(dst_pool, n_dst, src_pool, n_src, page_bytes, src, dst, n, done=None, stream=None) -> None:
    _check(lib().favor_pages_copy(_ptr(dst_pool), int(n_dst), _ptr(src_pool), int(n_src), int(page_bytes), _ptr(src),
                                  _ptr(dst), int(n), _ptr(done), _stream(stream, dst_pool)), "favor_pages_copy")


def favor_pages_clear(pool, n_pages, page_bytes, pages, n, stream=None) -> None:
    _check(lib().favor_pages_clear(_ptr(pool), int(n_pages), int(page_bytes), _ptr(pages), int(n),
                                   _stream(stream, pool)), "favor_pages_clear")


def favor_pages_compact(pool, n_pages, page_bytes, table, S, new_table, page_map, n_live, stream=None) -> None:
    _check(lib().favor_pages_compact(_ptr(pool), int(n_pages), int(page_bytes), _ptr(table), int(S), _ptr(new_table),
                                     _ptr(page_map), _ptr(n_live), _stream(stream, pool)), "favor_pages_compact")


def favor_pages_move(pool, n_pages, page_bytes, page_map, stream=None) -> None:
    _check(lib().favor_pages_move(_ptr(pool), int(n_pages), int(page_bytes), _ptr(page_map), _stream(stream, pool)),
           "favor_pages_move")


def _want(t, shape, dtype, device, name):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {list(shape)} on {device}, "
                         f"got {t.dtype} {list(t.shape)} on {t.device}")


class Ssm:
    """Owns one handle of the convolution and the scan; checks shapes, dtypes and devices before
    calling the C ABI.  Batches are token-major: [B, L, D], B and C [B, L, G, N]; a step call takes
    the same without L.  ``training=False`` leaves the backward calls' workspace out."""

    def __init__(self, D, N, G, K, dtype, max_B, max_L, training=True):
        import torch
        self.D, self.N, self.G, self.K = D, N, G, K
        self.dtype = dtype
        self.max_B, self.max_L = max_B, max_L
        self.handle = None
        self.handle = favor_ssm_create(D, N, G, K, dtype, max_B, max_L, training)
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._t = torch.float32 if DTYPE_CODES.get(dtype, dtype) == DTYPE_CODES["f32"] else torch.bfloat16

    # ---- checks
    def _seq(self, t, lead, name, optional=False):
        if t is None and optional:
            return
        _want(t, (*lead, self.D), self._t, self.device, name)

    def _par(self, t, shape, name, optional=True):
        import torch
        if t is None and optional:
            return
        _want(t, shape, torch.float32, self.device, name)

    def _int(self, t, n, name):
        import torch
        if t is not None:
            _want(t, (n,), torch.int32, self.device, name)

    def _pool(self, pool, page, dtype, name):
        """Number of pages of a pool (0: none given)."""
        if pool is None:
            return 0
        _want(pool, (pool.shape[0], *page), dtype, self.device, name)
        return pool.shape[0]

    @staticmethod
    def _lead(x, dims, name):
        if x.dim() != dims:
            raise ValueError(f"{name}: expected {dims} dimensions, got {list(x.shape)}")
        return tuple(x.shape[:-1])

    def _out(self, like, out, lens):
        """The output: rows behind a row's end are left as they are, so a new one starts at zero."""
        import torch
        if out is None:
            return torch.empty_like(like) if lens is None else torch.zeros_like(like)
        _want(out, like.shape, like.dtype, like.device, "out")
        return out

    # ---- states
    def new_state(self, P):
        """P empty scan states [P, D, N]."""
        import torch
        return torch.zeros((P, self.D, self.N), dtype=torch.float32, device=self.device)

    def new_window(self, P):
        """P empty convolution windows [P, K-1, D]."""
        import torch
        return torch.zeros((P, self.K - 1, self.D), dtype=self._t, device=self.device)

    # ---- convolution
    def conv(self, x, weight, bias=None, silu=True, window=None, pages=None, lens=None, out=None, stream=None):
        """The convolution of x [B, L, D]; with window (pages [P, K-1, D]) it continues each row's
        past and keeps the row's last inputs."""
        lead = self._lead(x, 3, "x")
        self._seq(x, lead, "x")
        self._par(weight, (self.D, self.K), "weight", optional=False)
        self._par(bias, (self.D,), "bias")
        P = self._pool(window, (self.K - 1, self.D), self._t, "window")
        self._int(pages, lead[0], "pages")
        self._int(lens, lead[0], "lens")
        out = self._out(x, out, lens)
        favor_conv_causal(self.handle, x, weight, bias, silu, window, pages, P, lens, out, *lead, stream)
        return out

    def conv_step(self, x, weight, window, bias=None, silu=True, pages=None, out=None, stream=None):
        """One token a row, x [B, D]; the rows' windows move on."""
        lead = self._lead(x, 2, "x")
        self._seq(x, lead, "x")
        self._par(weight, (self.D, self.K), "weight", optional=False)
        self._par(bias, (self.D,), "bias")
        P = self._pool(window, (self.K - 1, self.D), self._t, "window")
        self._int(pages, lead[0], "pages")
        out = self._out(x, out, None)
        favor_conv_causal_step(self.handle, x, weight, bias, silu, window, pages, P, out, *lead, stream)
        return out

    def conv_backward(self, x, weight, dout, bias=None, silu=True, lens=None, stream=None):
        """(dx, dweight, dbias) of conv(x, weight, bias, silu, lens=lens); dbias is None without bias."""
        import torch
        lead = self._lead(x, 3, "x")
        self._seq(x, lead, "x")
        self._seq(dout, lead, "dout")
        self._par(weight, (self.D, self.K), "weight", optional=False)
        self._par(bias, (self.D,), "bias")
        self._int(lens, lead[0], "lens")
        dx = self._out(x, None, lens)
        dweight = torch.empty_like(weight)
        dbias = None if bias is None else torch.empty_like(bias)
        favor_conv_causal_backward(self.handle, x, weight, bias, silu, lens, dout, dx, dweight, dbias, *lead, stream)
        return dx, dweight, dbias

    # ---- scan
    def _scan_args(self, lead, u, dt, A, Bm, Cm, skip, z, dt_bias):
        self._seq(u, lead, "u")
        self._seq(dt, lead, "dt")
        self._seq(z, lead, "z", optional=True)
        for t, name in ((Bm, "Bm"), (Cm, "Cm")):
            _want(t, (*lead, self.G, self.N), self._t, self.device, name)
        self._par(A, (self.D, self.N), "A", optional=False)
        self._par(skip, (self.D,), "skip")
        self._par(dt_bias, (self.D,), "dt_bias")

    def scan(self, u, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, state=None, pages=None, lens=None, out=None,
             stream=None):
        """The scan of u, dt [B, L, D]; with state (pages [P, D, N]) it continues each row's past and
        leaves the state behind the row's last token."""
        lead = self._lead(u, 3, "u")
        self._scan_args(lead, u, dt, A, Bm, Cm, skip, z, dt_bias)
        P = self._state(state)
        self._int(pages, lead[0], "pages")
        self._int(lens, lead[0], "lens")
        out = self._out(u, out, lens)
        favor_ssm_scan(self.handle, u, dt, A, Bm, Cm, skip, z, dt_bias, state, pages, P, lens, out, *lead, stream)
        return out

    def _state(self, state):
        import torch
        return self._pool(state, (self.D, self.N), torch.float32, "state")

    def scan_step(self, u, dt, A, Bm, Cm, state, skip=None, z=None, dt_bias=None, pages=None, out=None, stream=None):
        """One token a row: u, dt [B, D], Bm, Cm [B, G, N]; the rows' states move on."""
        lead = self._lead(u, 2, "u")
        self._scan_args(lead, u, dt, A, Bm, Cm, skip, z, dt_bias)
        P = self._state(state)
        self._int(pages, lead[0], "pages")
        out = self._out(u, out, None)
        favor_ssm_scan_step(self.handle, u, dt, A, Bm, Cm, skip, z, dt_bias, state, pages, P, out, *lead, stream)
        return out

    def scan_backward(self, u, dt, A, Bm, Cm, dout, skip=None, z=None, dt_bias=None, lens=None, stream=None):
        """Gradients of scan(u, dt, A, Bm, Cm, skip, z, dt_bias, lens=lens) for the upstream gradient
        dout, as a dict: du, ddt, dA, dB, dC, dskip, dz, ddt_bias (None where the input is None)."""
        import torch
        lead = self._lead(u, 3, "u")
        self._scan_args(lead, u, dt, A, Bm, Cm, skip, z, dt_bias)
        self._seq(dout, lead, "dout")
        self._int(lens, lead[0], "lens")
        new = torch.empty_like if lens is None else torch.zeros_like
        gr = dict(du=new(u), ddt=new(dt), dA=torch.empty_like(A), dB=new(Bm), dC=new(Cm),
                  dskip=None if skip is None else torch.empty_like(skip), dz=None if z is None else new(z),
                  ddt_bias=None if dt_bias is None else torch.empty_like(dt_bias))
        favor_ssm_scan_backward(self.handle, u, dt, A, Bm, Cm, skip, z, dt_bias, lens, dout, gr["du"], gr["ddt"],
                                gr["dA"], gr["dB"], gr["dC"], gr["dskip"], gr["dz"], gr["ddt_bias"], *lead, stream)
        return gr

    def close(self):
        if self.handle:
            favor_ssm_destroy(self.handle)
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


def _page_bytes(pool, name):
    if pool.dim() < 1 or pool.numel() == 0 or not pool.is_cuda or not pool.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous, non-empty CUDA tensor [pages, ...]")
    return pool[0].numel() * pool.element_size()


def _indices(t, device, name):
    import torch
    if t.dim() != 1 or t.numel() == 0 or t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous, non-empty int32 vector on {device}")


def _on(pool):
    import torch
    return torch.cuda.device(pool.device)


def pages_copy(dst_pool, src_pool, src, dst, stream=None):
    """dst_pool[dst[i]] = src_pool[src[i]] for every pair (the pools may be one tensor; a source named
    several times is forked).  Returns int32 [n]: 1 for a pair carried out, 0 for one left out (a
    page outside its pool, a destination named before, or, in one pool, one that the call reads)."""
    import torch
    pb = _page_bytes(dst_pool, "dst_pool")
    if _page_bytes(src_pool, "src_pool") != pb or src_pool.dtype != dst_pool.dtype \
            or src_pool.device != dst_pool.device:
        raise ValueError("the pools' pages differ in size, dtype or device")
    _indices(src, dst_pool.device, "src")
    _indices(dst, dst_pool.device, "dst")
    if src.numel() != dst.numel():
        raise ValueError(f"src names {src.numel()} pages and dst {dst.numel()}")
    done = torch.empty_like(src)
    with _on(dst_pool):
        favor_pages_copy(dst_pool, dst_pool.shape[0], src_pool, src_pool.shape[0], pb, src, dst, src.numel(), done,
                         stream)
    return done


def pages_clear(pool, pages, stream=None):
    """The named pages become the empty state (zeros); entries outside the pool are passed over."""
    pb = _page_bytes(pool, "pool")
    _indices(pages, pool.device, "pages")
    with _on(pool):
        favor_pages_clear(pool, pool.shape[0], pb, pages, pages.numel(), stream)


def pages_compact(pool, table, others=(), stream=None):
    """Move the pages that table names into the first pages of the pool, and the same pages of the
    ``others`` (pools of one cache share the table).  Returns (new_table, n_live): where each entry's
    page is now (-1 for an entry that names none), and the number of live pages, int32 [1]."""
    import torch
    pb = _page_bytes(pool, "pool")
    _indices(table, pool.device, "table")
    sizes = []
    for i, o in enumerate(others):
        sizes.append(_page_bytes(o, f"others[{i}]"))
        if o.shape[0] != pool.shape[0] or o.device != pool.device:
            raise ValueError(f"others[{i}]: expected {pool.shape[0]} pages on {pool.device}")
    new_table = torch.empty_like(table)
    n_live = torch.empty(1, dtype=torch.int32, device=pool.device)
    page_map = torch.empty(pool.shape[0], dtype=torch.int32, device=pool.device) if sizes else None
    with _on(pool):
        favor_pages_compact(pool, pool.shape[0], pb, table, table.numel(), new_table, page_map, n_live, stream)
        for o, ob in zip(others, sizes):
            favor_pages_move(o, o.shape[0], ob, page_map, stream)
    return new_table, n_live


def declare(L) -> None:
    """Argument types of the entry points above."""
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.favor_ssm_create.argtypes = [ctypes.POINTER(vp), i, i, i, i, i, i, i, i]
    L.favor_ssm_destroy.argtypes = [vp]
    L.favor_conv_causal.argtypes = [vp, vp, vp, vp, i, vp, vp, i, vp, vp, i, i, vp]
    L.favor_conv_causal_step.argtypes = [vp, vp, vp, vp, i, vp, vp, i, vp, i, vp]
    L.favor_conv_causal_backward.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, vp, vp, i, i, vp]
    L.favor_ssm_scan.argtypes = [vp] * 11 + [i, vp, vp, i, i, vp]
    L.favor_ssm_scan_step.argtypes = [vp] * 11 + [i, vp, i, vp]
    L.favor_ssm_scan_backward.argtypes = [vp] * 19 + [i, i, vp]
    L.favor_pages_copy.argtypes = [vp, i, vp, i, sz, vp, vp, i, vp, vp]
    L.favor_pages_clear.argtypes = [vp, i, sz, vp, i, vp]
    L.favor_pages_compact.argtypes = [vp, i, sz, vp, i, vp, vp, vp, vp]
    L.favor_pages_move.argtypes = [vp, i, sz, vp, vp]
    for name in __all__:
        if name.startswith("favor_"):
            getattr(L, name).restype = i
