"""Calls on an explicit stream: the tensors that a call makes for itself (outputs, gradients, tables,
their zero fills) belong to that stream's order.

The CPU tests run the binding with torch's stream calls and the library replaced by records; the GPU
tests keep the current stream busy with work that would overwrite an output made in its order."""
import contextlib
import types

import pytest
import torch

import random_feature_gb300 as R
from random_feature_gb300 import favor as _favor, ssm as _ssm

CUR, SIDE = 0x100, 0x200


class _Stream:
    def __init__(self, raw, *_, **__):
        self.cuda_stream = raw


class _Log:
    """The stream that is current, what was made on which, and what was told to the allocator."""

    def __init__(self):
        self.stack = [CUR]
        self.made, self.noted, self.calls = [], [], []


class _Made:
    """A tensor made by the call."""
    shape, dtype, device = (2,), None, None

    def __init__(self, log):
        self.log, self.at = log, log.stack[-1]
        log.made.append(self)

    def data_ptr(self):
        return 64

    def record_stream(self, s):
        self.log.noted.append((self, s.cuda_stream))

    def new_empty(self, *_):
        return _Made(self.log)


@pytest.fixture
def log(monkeypatch):
    log = _Log()

    @contextlib.contextmanager
    def current(s):
        log.stack.append(s.cuda_stream)
        yield
        log.stack.pop()

    for name in ("empty_like", "zeros_like", "empty", "zeros"):
        monkeypatch.setattr(torch, name, lambda *a, **k: _Made(log))
    monkeypatch.setattr(torch.cuda, "stream", current)
    # torch's takes the address 0 for "none given" and hands out one of its own streams
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, *a: _Stream(raw or 0x300))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: _Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Stream(log.stack[-1]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: log.stack[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                log.calls.append((name, args))
                return 0
            return call
    monkeypatch.setattr(_ssm, "lib", Lib)
    monkeypatch.setattr(_favor, "lib", Lib)
    log.lib = Lib()
    return log


def _ssm_object(log, D=4, N=8, K=2):
    f = object.__new__(R.Ssm)
    cpu = torch.device("cpu")
    f.D, f.N, f.G, f.K, f.handle, f.device, f._index = D, N, 1, K, None, cpu, 0
    f._t, f._f32, f._i32, f._lib = torch.float32, torch.float32, torch.int32, log.lib
    f._dims = (D,)
    f._weight, f._vec, f._A = ((D, K), torch.float32, cpu), ((D,), torch.float32, cpu), ((D, N), torch.float32, cpu)
    return f


def _ones(*shape, dtype=torch.float32):
    return torch.tensor(1, dtype=dtype).expand(shape).contiguous()


def _ssm_calls(f):
    B, L, D, N = 2, 3, f.D, f.N
    x, bc, A, w = _ones(B, L, D), _ones(B, L, 1, N), _ones(D, N), _ones(D, f.K)
    lens = _ones(B, dtype=torch.int32)
    state, win = _ones(B, D, N), _ones(B, f.K - 1, D)
    return {
        "conv": lambda s: f.conv(x, w, lens=lens, stream=s),
        "scan": lambda s: f.scan(x, x, A, bc, bc, lens=lens, stream=s),
        "conv_step": lambda s: f.conv_step(x[:, 0].contiguous(), w, win, stream=s),
        "scan_step": lambda s: f.scan_step(x[:, 0].contiguous(), x[:, 0].contiguous(), A, bc[:, 0].contiguous(),
                                           bc[:, 0].contiguous(), state, stream=s),
        "conv_backward": lambda s: f.conv_backward(x, w, x, A[:, 0].contiguous(), stream=s),
        "scan_backward": lambda s: f.scan_backward(x, x, A, bc, bc, x, skip=A[:, 0].contiguous(), z=x, stream=s),
    }


SSM = ("conv", "scan", "conv_step", "scan_step", "conv_backward", "scan_backward")


@pytest.mark.parametrize("given", [SIDE, _Stream(SIDE)], ids=["address", "object"])
@pytest.mark.parametrize("call", SSM)
def test_ssm_outputs_belong_to_the_given_stream(log, call, given):
    _ssm_calls(_ssm_object(log))[call](given)
    assert log.made and all(t.at == SIDE for t in log.made)
    assert len(log.calls) == 1 and log.calls[0][1][-1] == SIDE
    # the current stream may read them until they are freed
    assert log.noted == [(t, CUR) for t in log.made]


@pytest.mark.parametrize("given", [0, 1, _Stream(0)], ids=["address", "second-name", "object"])
@pytest.mark.parametrize("call", SSM)
def test_ssm_outputs_on_the_default_stream(log, call, given):
    _ssm_calls(_ssm_object(log))[call](given)
    assert log.made and all(t.at == 0 for t in log.made)
    assert log.noted == [(t, CUR) for t in log.made]


@pytest.mark.parametrize("given", [None, CUR, _Stream(CUR)], ids=["none", "address", "object"])
@pytest.mark.parametrize("call", SSM)
def test_ssm_outputs_on_the_current_stream(log, call, given):
    _ssm_calls(_ssm_object(log))[call](given)
    assert log.made and all(t.at == CUR for t in log.made) and not log.noted
    assert len(log.calls) == 1 and log.calls[0][1][-1] == CUR


@pytest.mark.parametrize("given", [SIDE, None])
def test_page_tables_belong_to_the_given_stream(log, monkeypatch, given):
    pool = types.SimpleNamespace(numel=lambda: 8, dim=lambda: 2, is_cuda=True, is_contiguous=lambda: True, shape=(4, 2),
                                 element_size=lambda: 4, get_device=lambda: 0, data_ptr=lambda: 64, dtype=None)

    class Index(_Made):
        dtype, shape = torch.int32, (2,)
        dim, numel, get_device = (lambda s: 1), (lambda s: 2), (lambda s: 0)
        is_contiguous = lambda s: True
    idx = Index(log)
    log.made.clear()
    want = SIDE if given else CUR
    R.pages_copy(pool, pool, idx, idx, stream=given)
    R.pages_compact(pool, idx, others=(pool,), stream=given)
    assert len(log.made) == 4 and all(t.at == want for t in log.made)
    assert [c[1][-1] for c in log.calls] == [want] * 3
    # page_map is not handed out: it needs no note, but may have one
    assert all(s == CUR for _, s in log.noted) and len(log.noted) >= (3 if given else 0)


FAVOR = {
    "feature_map": lambda f, t, s: f.feature_map(t, stream=s),
    "attn": lambda f, t, s: f.attn(t, t, t, stream=s),
    "attn_causal": lambda f, t, s: f.attn(t, t, t, causal=True, stream=s),
    "attn_backward": lambda f, t, s: f.attn_backward(t, t, t, t, stream=s),
    "attn_causal_gated": lambda f, t, s: f.attn_causal_gated(t, t, t, t.gate, stream=s),
    "causal_step_gated": lambda f, t, s: f.causal_step_gated(t, t, t, t.gate, t, stream=s),
    "kv_state": lambda f, t, s: f.kv_state(t, t, stream=s),
    "attn_from_state": lambda f, t, s: f.attn_from_state(t, t, stream=s),
    "causal_step": lambda f, t, s: f.causal_step(t, t, t, t, stream=s),
}


@pytest.mark.parametrize("given", [SIDE, None])
@pytest.mark.parametrize("call", FAVOR)
def test_favor_outputs_belong_to_the_given_stream(log, call, given):
    f = object.__new__(R.Favor)
    f.H, f.m, f.d, f.dv, f.dtype, f.handle = 2, 8, 4, 4, "f32", None
    f._chk = f._chk_state = lambda *a: None
    yes = lambda: True
    gate = types.SimpleNamespace(shape=(1, 2, 3), dtype=torch.float32, is_cuda=True, is_contiguous=yes,
                                 data_ptr=lambda: 64)
    t = types.SimpleNamespace(shape=(1, 2, 3, 4), device=None, data_ptr=lambda: 64, gate=gate)
    FAVOR[call](f, t, given)
    want = SIDE if given else CUR
    assert log.made and all(m.at == want for m in log.made)
    assert log.noted == [(m, CUR) for m in log.made if given]
    assert len(log.calls) == 1 and log.calls[0][1][-1] == want


# ---- on the GPU
def _busy(seconds=0.15):
    """Ordinary work of about that time on the current stream, without waiting for it."""
    a = torch.full((4096, 4096), 1e-3, device="cuda", dtype=torch.bfloat16)
    b = torch.empty_like(a)
    torch.mm(a, a, out=b)
    torch.cuda.synchronize()
    for _ in range(int(seconds / 1e-4)):        # 1.4e11 operations: 0.07 ms at least
        torch.mm(a, a, out=b)


def _later_writes(shapes):
    """Blocks of those sizes, freed on the current stream with writes to them still queued there: what
    the allocator hands out in that stream's order next."""
    for shape, dtype in shapes:
        for _ in range(2):
            t = torch.empty(shape, dtype=dtype, device="cuda")
            t.fill_(77)
            del t


def _gpu_case():
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=g)
    B, L, D, N = 3, 200, 96, 16
    t = dict(x=rn(B, L, D), dt=rn(B, L, D), z=rn(B, L, D), dout=rn(B, L, D), Bm=rn(B, L, 1, N), Cm=rn(B, L, 1, N),
             A=-torch.exp(rn(D, N)), skip=rn(D), w=rn(D, 4), bias=rn(D))
    t["lens"] = torch.tensor([200, 0, 77], dtype=torch.int32, device="cuda")
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("as_address", [True, False])
@pytest.mark.parametrize("call", SSM)
def test_ssm_calls_beside_a_busy_stream(call, as_address):
    t = _gpu_case()
    B, L, D = t["x"].shape
    N = t["A"].shape[1]
    with R.Ssm(D, N, 1, 4, "f32", B, L) as f:
        tok = {k: v[:, 0].contiguous() for k, v in t.items() if v.dim() > 2}
        win, state = f.new_window(B), f.new_state(B)
        run = {
            "conv": lambda s: (f.conv(t["x"], t["w"], t["bias"], lens=t["lens"], stream=s),),
            "scan": lambda s: (f.scan(t["x"], t["dt"], t["A"], t["Bm"], t["Cm"], t["skip"], t["z"], lens=t["lens"],
                                      stream=s),),
            "conv_step": lambda s: (f.conv_step(tok["x"], t["w"], win.zero_() if s is None else win, stream=s),),
            "scan_step": lambda s: (f.scan_step(tok["x"], tok["dt"], t["A"], tok["Bm"], tok["Cm"],
                                                state.zero_() if s is None else state, stream=s),),
            "conv_backward": lambda s: f.conv_backward(t["x"], t["w"], t["dout"], t["bias"], lens=t["lens"], stream=s),
            "scan_backward": lambda s: tuple(v for v in f.scan_backward(
                t["x"], t["dt"], t["A"], t["Bm"], t["Cm"], t["dout"], skip=t["skip"], z=t["z"], lens=t["lens"],
                stream=s).values() if v is not None),
        }[call]
        want = [v.clone() for v in run(None)]
        win.zero_(), state.zero_()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        _busy()
        _later_writes([(v.shape, v.dtype) for v in want])
        got = run(side.cuda_stream if as_address else side)
        side.synchronize()
        assert not torch.cuda.current_stream().query()      # the work there was still going on
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["kv_state", "attn_causal", "attn_backward"])
def test_favor_calls_beside_a_busy_stream(call):
    import numpy as np
    B, H, L, d, m = 2, 2, 130, 16, 32
    omega = np.random.default_rng(2).standard_normal((H, m, d)).astype(np.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, do = (0.5 * torch.randn(B, H, L, d, device="cuda", generator=g) for _ in range(4))
    with R.Favor(H, m, d, d, "softmax_pos", "f32", omega, 0.5, B, L) as f:
        run = {"kv_state": lambda s: (f.kv_state(k, v, stream=s),),
               "attn_causal": lambda s: (f.attn(q, k, v, causal=True, stream=s),),
               "attn_backward": lambda s: f.attn_backward(q, k, v, do, stream=s)}[call]
        want = [t.clone() for t in run(None)]
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        _busy()
        _later_writes([(t.shape, t.dtype) for t in want])
        got = run(side)
        side.synchronize()
        assert not torch.cuda.current_stream().query()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("given", [0, 1, "object"])
def test_calls_on_the_default_stream_beside_a_busy_current_one(given):
    t = _gpu_case()
    B, L, D = t["x"].shape
    if given == "object":
        given = torch.cuda.default_stream()
    with R.Ssm(D, 16, 1, 4, "f32", B, L) as f:
        run = lambda s: f.scan(f.conv(t["x"], t["w"], t["bias"], lens=t["lens"], stream=s), t["dt"], t["A"], t["Bm"],
                               t["Cm"], lens=t["lens"], stream=s)
        want = run(None).clone()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            _busy()
            _later_writes([(want.shape, want.dtype)])
            got = run(given)
            torch.cuda.default_stream().synchronize()
            assert not side.query()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.gpu
def test_outputs_freed_while_the_current_stream_reads_them():
    """An output made on another stream and dropped while the current stream still has to read it is not
    handed out again before that."""
    t = _gpu_case()
    B, L, D = t["x"].shape
    with R.Ssm(D, 16, 1, 4, "f32", B, L) as f:
        want = f.conv(t["x"], t["w"], t["bias"]).clone()
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        out = f.conv(t["x"], t["w"], t["bias"], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        _busy()
        copy = out.clone()
        del out
        for _ in range(4):
            f.conv(t["dout"], t["w"], t["bias"], stream=side)
        torch.cuda.synchronize()
        assert torch.equal(copy, want)


@pytest.mark.gpu
def test_page_calls_beside_a_busy_stream():
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    pool = torch.arange(12 * 64, device="cuda", dtype=torch.float32).view(12, 64)
    win = torch.arange(12 * 3, device="cuda", dtype=torch.float32).view(12, 3)
    src, dst, table = ints([1, 1, 20]), ints([5, 6, 7]), ints([11, 3, -1, 8])
    side = torch.cuda.Stream()
    # a kernel's first launch loads it, which waits for the device: launch each of them once before
    shapes = [((3,), torch.int32), ((4,), torch.int32), ((1,), torch.int32), ((12,), torch.int32)]
    _later_writes(shapes)
    other = pool.clone(), win.clone()
    R.pages_copy(other[0], other[0], src, dst)
    R.pages_compact(other[0], table, others=[other[1]])
    torch.cuda.synchronize()
    _busy()
    _later_writes(shapes)
    done = R.pages_copy(pool, pool, src, dst, stream=side)
    new, live = R.pages_compact(pool, table, others=[win], stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert done.tolist() == [1, 1, 0] and live.tolist() == [3]
    # live pages 3, 8, 11 (U = 3): they move, in order, to pages 0, 1, 2
    assert new.tolist() == [2, 0, -1, 1]
    for p, old in enumerate((3, 8, 11)):
        assert torch.equal(win[p], torch.arange(old * 3, old * 3 + 3, device="cuda", dtype=torch.float32))
        assert torch.equal(pool[p], torch.arange(old * 64, old * 64 + 64, device="cuda", dtype=torch.float32))


@pytest.mark.gpu
def test_a_captured_call_on_a_stream_beside_the_capturing_one():
    """A capture that forks to another stream by the calls' own argument, replayed on other inputs."""
    t = _gpu_case()
    B, L, D = t["x"].shape
    with R.Ssm(D, 16, 1, 4, "f32", B, L) as f:
        def block(x, s):
            u = f.conv(x, t["w"], t["bias"], lens=t["lens"], stream=s)
            return f.scan(u, t["dt"], t["A"], t["Bm"], t["Cm"], lens=t["lens"], stream=s)
        want = [block(t[k], None).clone() for k in ("x", "dout")]
        inp, side = t["x"].clone(), torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            out = block(inp, side)
            main.wait_stream(side)
        for k, w in zip(("x", "dout"), want):
            inp.copy_(t[k])
            graph.replay()
            assert torch.equal(out, w)
