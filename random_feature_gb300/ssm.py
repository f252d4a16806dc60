"""ctypes binding of the selective scan, the short causal convolution and the state
pages of the C ABI (include/favor.h).

Like the attention binding: argument marshalling and checks only, the functions
keep the C names, the stream defaults to torch's current stream on the tensor's
device, and nothing falls back to anything when the library is missing.
"""
from __future__ import annotations

import ctypes
from operator import attrgetter

from .favor import DTYPE_CODES, _check, _made_on, _ptr, _stream, lib

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


def _raw_stream(stream, index):
    """The stream's address; torch's current one on the device by default.  (Looked up without building
    a stream object: a decoding step's host time is mostly such calls.)"""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


_kind = attrgetter("shape", "dtype", "device")


def _at(t):
    return None if t is None else t.data_ptr()


class Ssm:
    """Owns one handle of the convolution and the scan; checks shapes, dtypes and devices before
    calling the C ABI.  Batches are token-major: [B, L, D], B and C [B, L, G, N]; a step call takes
    the same without L.  ``training=False`` leaves the backward calls' workspace out.

    ``scan`` and the backward calls use the handle's workspace: of one object, such calls (and
    replays of graphs that hold them) must not overlap on the device; use an object a stream.
    Several host threads may call one object on one stream.
    ``conv``, the step calls and the page functions use none.

    A call with ``stream`` makes its outputs in that stream's order; that the inputs are ready there, and
    that whoever reads the outputs on another stream waits for the call, is the caller's to arrange."""

    def __init__(self, D, N, G, K, dtype, max_B, max_L, training=True):
        import torch
        self.D, self.N, self.G, self.K = D, N, G, K
        self.dtype = dtype
        self.max_B, self.max_L = max_B, max_L
        self.handle = None
        self.handle = favor_ssm_create(D, N, G, K, dtype, max_B, max_L, training)
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self._t = torch.float32 if DTYPE_CODES.get(dtype, dtype) == DTYPE_CODES["f32"] else torch.bfloat16
        self._f32, self._i32, self._lib = torch.float32, torch.int32, lib()

        # what the parameters have to be: shape, dtype, device
        f32 = torch.float32
        self._dims = (D,)
        self._weight, self._vec, self._A = (((D, K), f32, self.device), ((D,), f32, self.device),
                                            ((D, N), f32, self.device))

    # ---- checks
    def _check_all(self, items):
        """Every tensor of (tensor or None, (shape, dtype, device), name)."""
        for t, want, name in items:
            if t is not None and (_kind(t) != want or not t.is_contiguous()):
                raise ValueError(f"{name}: expected contiguous {want[1]} {list(want[0])} on {want[2]}, "
                                 f"got {t.dtype} {list(t.shape)} on {t.device}")

    def _pool(self, pool, page, dtype, name):
        """(number of pages, what the pool has to be)."""
        if pool is None:
            return 0, None
        P = pool.shape[0] if pool.dim() else 0
        if P == 0:      # its address is NULL, which means that there is none
            raise ValueError(f"{name}: expected at least one page {list(page)}, got {list(pool.shape)}")
        return P, ((P, *page), dtype, self.device)

    @staticmethod
    def _lead(x, dims, name):
        if x.dim() != dims:
            raise ValueError(f"{name}: expected {dims} dimensions, got {list(x.shape)}")
        return tuple(x.shape[:-1])

    def _out(self, like, out, stream, lens=None):
        """The output: rows behind a row's end are left as they are, so a new one starts at zero."""
        if out is None:
            import torch
            new = torch.empty_like if lens is None else torch.zeros_like
            return new(like) if stream is None else _made_on(stream, self.device, lambda: new(like))
        self._check_all(((out, _kind(like), "out"),))
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
    def _conv_args(self, lead, x, weight, bias, window, pages, lens):
        """Checks; the number of window pages."""
        P, pool = self._pool(window, (self.K - 1, self.D), self._t, "window")
        rows = (lead[:1], self._i32, self.device)
        self._check_all(((x, (lead + self._dims, self._t, self.device), "x"), (weight, self._weight, "weight"),
                         (bias, self._vec, "bias"), (window, pool, "window"), (pages, rows, "pages"),
                         (lens, rows, "lens")))
        return P

    def conv(self, x, weight, bias=None, silu=True, window=None, pages=None, lens=None, out=None, stream=None):
        """The convolution of x [B, L, D]; with window (pages [P, K-1, D]) it continues each row's
        past and keeps the row's last inputs."""
        B, L = lead = self._lead(x, 3, "x")
        P = self._conv_args(lead, x, weight, bias, window, pages, lens)
        out = self._out(x, out, stream, lens)
        _check(self._lib.favor_conv_causal(self.handle, x.data_ptr(), weight.data_ptr(), _at(bias), int(silu),
                                           _at(window), _at(pages), P, _at(lens), out.data_ptr(), B, L,
                                           _raw_stream(stream, self._index)), "favor_conv_causal")
        return out

    def conv_step(self, x, weight, window, bias=None, silu=True, pages=None, out=None, stream=None):
        """One token a row, x [B, D]; the rows' windows move on."""
        lead = self._lead(x, 2, "x")
        P = self._conv_args(lead, x, weight, bias, window, pages, None)
        out = self._out(x, out, stream)
        _check(self._lib.favor_conv_causal_step(self.handle, x.data_ptr(), weight.data_ptr(), _at(bias), int(silu),
                                                _at(window), _at(pages), P, out.data_ptr(), lead[0],
                                                _raw_stream(stream, self._index)), "favor_conv_causal_step")
        return out

    def conv_backward(self, x, weight, dout, bias=None, silu=True, lens=None, stream=None):
        """(dx, dweight, dbias) of conv(x, weight, bias, silu, lens=lens); dbias is None without bias."""
        import torch
        B, L = lead = self._lead(x, 3, "x")
        self._conv_args(lead, x, weight, bias, None, None, lens)
        self._check_all(((dout, _kind(x), "dout"),))
        new = torch.empty_like
        dx, dweight, dbias = _made_on(stream, self.device,
                                      lambda: (new(x), new(weight), None if bias is None else new(bias)))
        _check(self._lib.favor_conv_causal_backward(self.handle, x.data_ptr(), weight.data_ptr(), _at(bias), int(silu),
                                                    _at(lens), dout.data_ptr(), dx.data_ptr(), dweight.data_ptr(),
                                                    _at(dbias), B, L, _raw_stream(stream, self._index)),
               "favor_conv_causal_backward")
        return dx, dweight, dbias

    # ---- scan
    def _scan_args(self, lead, u, dt, A, Bm, Cm, skip, z, dt_bias, state, pages, lens):
        """Checks; the number of state pages."""
        dev = self.device
        P, pool = self._pool(state, (self.D, self.N), self._f32, "state")
        seq, mat = (lead + self._dims, self._t, dev), (lead + (self.G, self.N), self._t, dev)
        rows = (lead[:1], self._i32, dev)
        self._check_all(((u, seq, "u"), (dt, seq, "dt"), (z, seq, "z"), (Bm, mat, "Bm"), (Cm, mat, "Cm"),
                         (A, self._A, "A"), (skip, self._vec, "skip"), (dt_bias, self._vec, "dt_bias"),
                         (state, pool, "state"), (pages, rows, "pages"), (lens, rows, "lens")))
        return P

    def scan(self, u, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, state=None, pages=None, lens=None, out=None,
             stream=None):
        """The scan of u, dt [B, L, D]; with state (pages [P, D, N]) it continues each row's past and
        leaves the state behind the row's last token."""
        B, L = lead = self._lead(u, 3, "u")
        P = self._scan_args(lead, u, dt, A, Bm, Cm, skip, z, dt_bias, state, pages, lens)
        out = self._out(u, out, stream, lens)
        _check(self._lib.favor_ssm_scan(self.handle, u.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(),
                                        Cm.data_ptr(), _at(skip), _at(z), _at(dt_bias), _at(state), _at(pages), P,
                                        _at(lens), out.data_ptr(), B, L, _raw_stream(stream, self._index)),
               "favor_ssm_scan")
        return out

    def scan_step(self, u, dt, A, Bm, Cm, state, skip=None, z=None, dt_bias=None, pages=None, out=None, stream=None):
        """One token a row: u, dt [B, D], Bm, Cm [B, G, N]; the rows' states move on."""
        lead = self._lead(u, 2, "u")
        P = self._scan_args(lead, u, dt, A, Bm, Cm, skip, z, dt_bias, state, pages, None)
        out = self._out(u, out, stream)
        _check(self._lib.favor_ssm_scan_step(self.handle, u.data_ptr(), dt.data_ptr(), A.data_ptr(), Bm.data_ptr(),
                                             Cm.data_ptr(), _at(skip), _at(z), _at(dt_bias), _at(state), _at(pages),
                                             P, out.data_ptr(), lead[0], _raw_stream(stream, self._index)),
               "favor_ssm_scan_step")
        return out

    def scan_backward(self, u, dt, A, Bm, Cm, dout, skip=None, z=None, dt_bias=None, lens=None, stream=None):
        """Gradients of scan(u, dt, A, Bm, Cm, skip, z, dt_bias, lens=lens) for the upstream gradient
        dout, as a dict: du, ddt, dA, dB, dC, dskip, dz, ddt_bias (None where the input is None)."""
        import torch
        B, L = lead = self._lead(u, 3, "u")
        self._scan_args(lead, u, dt, A, Bm, Cm, skip, z, dt_bias, None, None, lens)
        self._check_all(((dout, _kind(u), "dout"),))
        new = torch.empty_like
        gr = dict(zip(("du", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias"), _made_on(
            stream, self.device,
            lambda: tuple(None if t is None else new(t) for t in (u, dt, A, Bm, Cm, skip, z, dt_bias)))))
        _check(self._lib.favor_ssm_scan_backward(self.handle, u.data_ptr(), dt.data_ptr(), A.data_ptr(),
                                                 Bm.data_ptr(), Cm.data_ptr(), _at(skip), _at(z), _at(dt_bias),
                                                 _at(lens), dout.data_ptr(), *(_at(g) for g in gr.values()), B, L,
                                                 _raw_stream(stream, self._index)), "favor_ssm_scan_backward")
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
    n = pool.numel()
    if n == 0 or pool.dim() < 1 or not pool.is_cuda or not pool.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous, non-empty CUDA tensor [pages, ...]")
    return n // pool.shape[0] * pool.element_size()


def _indices(t, index, name):
    import torch
    if t.dim() != 1 or t.numel() == 0 or t.dtype is not torch.int32 or t.get_device() != index \
            or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous, non-empty int32 vector on cuda:{index}")


def _on(index, call):
    """call() with the device current."""
    import torch
    if torch._C._cuda_getDevice() == index:
        return call()
    with torch.cuda.device(index):
        return call()


def pages_copy(dst_pool, src_pool, src, dst, stream=None):
    """dst_pool[dst[i]] = src_pool[src[i]] for every pair (the pools may be one tensor; a source named
    several times is forked).  Returns int32 [n]: 1 for a pair carried out, 0 for one left out (a
    page outside its pool, a destination named before, or, in one pool, one that the call reads)."""
    import torch
    pb, index = _page_bytes(dst_pool, "dst_pool"), dst_pool.get_device()
    if src_pool is not dst_pool and (_page_bytes(src_pool, "src_pool") != pb or src_pool.dtype is not dst_pool.dtype
                                     or src_pool.get_device() != index):
        raise ValueError("the pools' pages differ in size, dtype or device")
    _indices(src, index, "src")
    _indices(dst, index, "dst")
    n = src.shape[0]
    if n != dst.shape[0]:
        raise ValueError(f"src names {n} pages and dst {dst.shape[0]}")
    done = _made_on(stream, src.device, lambda: torch.empty_like(src))
    _check(_on(index, lambda: lib().favor_pages_copy(dst_pool.data_ptr(), dst_pool.shape[0], src_pool.data_ptr(),
                                                     src_pool.shape[0], pb, src.data_ptr(), dst.data_ptr(), n,
                                                     done.data_ptr(), _raw_stream(stream, index))),
           "favor_pages_copy")
    return done


def pages_clear(pool, pages, stream=None):
    """The named pages become the empty state (zeros); entries outside the pool are passed over."""
    pb, index = _page_bytes(pool, "pool"), pool.get_device()
    _indices(pages, index, "pages")
    _check(_on(index, lambda: lib().favor_pages_clear(pool.data_ptr(), pool.shape[0], pb, pages.data_ptr(),
                                                      pages.shape[0], _raw_stream(stream, index))),
           "favor_pages_clear")


def pages_compact(pool, table, others=(), stream=None):
    """Move the pages that table names into the first pages of the pool, and the same pages of the
    ``others`` (pools of one cache share the table).  Returns (new_table, n_live): where each entry's
    page is now (-1 for an entry that names none), and the number of live pages, int32 [1]."""
    import torch
    pb, index, P = _page_bytes(pool, "pool"), pool.get_device(), pool.shape[0]
    _indices(table, index, "table")
    others = tuple(others)      # walked twice
    sizes = []
    for i, o in enumerate(others):
        sizes.append(_page_bytes(o, f"others[{i}]"))
        if o.shape[0] != P or o.get_device() != index:
            raise ValueError(f"others[{i}]: expected {P} pages on cuda:{index}")
    new_table, n_live, page_map = _made_on(stream, table.device, lambda: (
        torch.empty_like(table), table.new_empty(1), table.new_empty(P) if sizes else None))

    def call():
        s = _raw_stream(stream, index)
        _check(lib().favor_pages_compact(pool.data_ptr(), P, pb, table.data_ptr(), table.shape[0],
                                         new_table.data_ptr(), _at(page_map), n_live.data_ptr(), s),
               "favor_pages_compact")
        for o, ob in zip(others, sizes):
            _check(lib().favor_pages_move(o.data_ptr(), P, ob, page_map.data_ptr(), s), "favor_pages_move")

    _on(index, call)
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
