"""Refusals of the scan, convolution and page calls that need no GPU: every argument check runs on
the host before anything is launched."""
import ctypes

import pytest

import random_feature_gb300 as R
from random_feature_gb300 import build as _build

BAD, UNS = R.FAVOR_ERR_INVALID_ARG, R.FAVOR_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def _built_library():
    _build.build()


@pytest.mark.parametrize("kw,want", [
    (dict(D=0), BAD), (dict(N=0), BAD), (dict(G=0), BAD), (dict(K=0), BAD), (dict(max_B=0), BAD), (dict(max_L=0), BAD),
    (dict(dtype=2), BAD), (dict(G=3), BAD), (dict(N=12), UNS), (dict(N=128), UNS), (dict(K=1), UNS), (dict(K=5), UNS),
    (dict(D=1 << 21), UNS), (dict(max_B=1 << 16, max_L=1 << 15), UNS), (dict(D=1 << 20, max_L=1 << 20), UNS),
    (dict(D=1 << 20, max_B=1 << 11, max_L=1), UNS), (dict(D=1 << 16, G=1 << 16, max_B=8, max_L=1 << 14), UNS),
])
def test_create_refuses(kw, want):
    a = {**dict(D=64, N=16, G=1, K=4, dtype=0, max_B=2, max_L=128), **kw}
    h = ctypes.c_void_p(12345)
    n0 = R.favor_launch_count()
    st = R.lib().favor_ssm_create(ctypes.byref(h), a["D"], a["N"], a["G"], a["K"], a["dtype"], a["max_B"], a["max_L"], 1)
    assert st == want, R.favor_last_error()
    assert h.value is None and R.favor_last_error() and R.favor_launch_count() == n0


def test_null_handles():
    L = R.lib()
    assert L.favor_ssm_create(None, 64, 16, 1, 4, 0, 1, 1, 1) == BAD
    assert L.favor_conv_causal(None, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, None) == BAD
    assert L.favor_conv_causal_step(None, 1, 1, 1, 1, 1, 1, 1, 1, 1, None) == BAD
    assert L.favor_conv_causal_backward(None, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, None) == BAD
    assert L.favor_ssm_scan(None, *[1] * 15, None) == BAD
    assert L.favor_ssm_scan_step(None, *[1] * 13, None) == BAD
    assert L.favor_ssm_scan_backward(None, *[1] * 20, None) == BAD
    assert L.favor_ssm_destroy(None) == R.FAVOR_OK


MB = 1 << 20


@pytest.mark.parametrize("call,want", [
    (lambda L: L.favor_pages_copy(None, 4, MB, 4, 16, 1, 1, 1, None, None), BAD),
    (lambda L: L.favor_pages_copy(MB, 0, MB, 4, 16, 4, 4, 1, None, None), BAD),
    (lambda L: L.favor_pages_copy(MB, 4, 2 * MB, 4, 0, 4, 4, 1, None, None), BAD),
    (lambda L: L.favor_pages_copy(MB, 4, 2 * MB, 4, 16, None, 4, 1, None, None), BAD),
    (lambda L: L.favor_pages_copy(MB, 4, 2 * MB, 4, 16, 4, 4, 0, None, None), BAD),
    (lambda L: L.favor_pages_copy(MB, 4, MB + 32, 4, 16, 4, 4, 1, None, None), BAD),      # pools overlap in part
    (lambda L: L.favor_pages_copy(MB, 1 << 30, 2 * MB, 4, 1 << 20, 4, 4, 1, None, None), UNS),
    (lambda L: L.favor_pages_clear(None, 4, 16, 4, 1, None), BAD),
    (lambda L: L.favor_pages_clear(MB, 4, 16, None, 1, None), BAD),
    (lambda L: L.favor_pages_clear(MB, 4, 16, 4, 0, None), BAD),
    (lambda L: L.favor_pages_compact(None, 4, 16, 4, 1, 64, None, 128, None), BAD),
    (lambda L: L.favor_pages_compact(MB, 4, 16, None, 1, 64, None, 128, None), BAD),
    (lambda L: L.favor_pages_compact(MB, 4, 16, 4, 0, 64, None, 128, None), BAD),
    (lambda L: L.favor_pages_compact(MB, 4, 16, 64, 3, 72, None, 128, None), BAD),        # table and new_table overlap
    (lambda L: L.favor_pages_compact(MB, 4, 16, 64, 3, 96, 100, 128, None), BAD),         # new_table and page_map
    (lambda L: L.favor_pages_compact(MB, (1 << 17) + 1, 16, 4, 1, 64, None, 128, None), UNS),
    (lambda L: L.favor_pages_copy(MB, 4, 2 * MB, 4, 16, 6, 4, 1, None, None), BAD),       # index off its element
    (lambda L: L.favor_pages_copy(MB, 4, 2 * MB, 4, 16, MB + 8, 4, 1, None, None), BAD),  # indices in the pool
    (lambda L: L.favor_pages_copy(MB, 4, 2 * MB, 4, 16, 64, 128, 2, 132, None), BAD),     # done over dst
    (lambda L: L.favor_pages_clear(MB, 4, 16, MB + 4, 1, None), BAD),
    (lambda L: L.favor_pages_clear(MB, 4, 16, 5, 1, None), BAD),
    (lambda L: L.favor_pages_compact(MB, 4, 16, MB, 1, 64, None, 128, None), BAD),
    (lambda L: L.favor_pages_compact(MB, 4, 16, 6, 1, 64, None, 128, None), BAD),
    (lambda L: L.favor_pages_move(MB, 4, 16, MB + 4, None), BAD),
    (lambda L: L.favor_pages_move(MB, 4, 16, 7, None), BAD),
    (lambda L: L.favor_pages_move(None, 4, 16, 4, None), BAD),
    (lambda L: L.favor_pages_move(MB, 4, 16, None, None), BAD),
])
def test_page_calls_refuse(call, want):
    n0 = R.favor_launch_count()
    assert call(R.lib()) == want, R.favor_last_error()
    assert R.favor_last_error() and R.favor_launch_count() == n0


@pytest.mark.gpu
def test_calls_refuse():
    """Bad calls on a good handle: refused before any launch, the tensors untouched."""
    import torch
    D, N, B, L = 32, 16, 2, 12
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")
    f4 = torch.float32
    u, bc, A, w = t(B, L, D), t(B, L, 1, N), t(D, N, dtype=f4), t(D, 4, dtype=f4)
    with R.Ssm(D, N, 1, 4, "bf16", B, L, training=False) as f:
        st, win = f.new_state(B), f.new_window(B)
        n0 = R.favor_launch_count()
        for bad in (lambda: f.scan(u.float(), u, A, bc, bc), lambda: f.scan(u, u[:, :5], A, bc, bc),
                    lambda: f.scan(u, u, A.bfloat16(), bc, bc), lambda: f.scan(u, u, A, bc[..., :8], bc),
                    lambda: f.scan(u, u, A, bc, bc, state=st.bfloat16()), lambda: f.scan(u, u, A.cpu(), bc, bc),
                    lambda: f.scan(u, u, A, bc, bc, lens=torch.zeros(B, device="cuda")),
                    lambda: f.scan(u, u, A, bc, bc, state=st, pages=torch.zeros(B + 1, dtype=torch.int32, device="cuda")),
                    lambda: f.scan(u.transpose(1, 2), u, A, bc, bc), lambda: f.scan(u[0], u, A, bc, bc),
                    lambda: f.conv(u, w[:, :3]), lambda: f.conv(u, w, window=win[:, :2]),
                    lambda: f.conv_step(u, w, win), lambda: f.conv(u, w, out=torch.empty_like(u)[:, :3]),
                    lambda: R.pages_copy(st, win, t(1, dtype=torch.int32), t(1, dtype=torch.int32)),
                    lambda: R.pages_copy(st, st, t(1, dtype=torch.int32), t(2, dtype=torch.int32)),
                    lambda: R.pages_clear(st, t(1, dtype=torch.int64)), lambda: R.pages_clear(st[:, ::2], t(1, dtype=torch.int32)),
                    lambda: R.pages_compact(st, t(0, dtype=torch.int32)),
                    lambda: R.pages_compact(st, t(1, dtype=torch.int32), others=[win[:1]])):
            with pytest.raises(ValueError):
                bad()
        one = f.new_state(1)
        for bad, status in ((lambda: f.scan(u, u, A, bc, bc, out=u), BAD),                      # out over an input
                            (lambda: f.conv(u, w, out=u), BAD),
                            (lambda: f.scan(u, u, A, bc, bc, state=one), BAD),                  # too few pages
                            (lambda: f.scan(u, u, A, bc, bc, pages=t(B, dtype=torch.int32)), BAD),   # pages, no state
                            (lambda: f.scan(t(B + 1, L, D), t(B + 1, L, D), A, t(B + 1, L, 1, N), t(B + 1, L, 1, N)), BAD),
                            (lambda: f.conv(t(B, L + 1, D), w), BAD),
                            (lambda: f.scan_backward(u, u, A, bc, bc, u), UNS),                 # no training workspace
                            (lambda: f.conv_backward(u, w, u), UNS)):
            with pytest.raises(R.FavorError) as e:
                bad()
            assert e.value.status == status, str(e.value)
        with pytest.raises(R.FavorError) as e:      # the state's pages are read 16 bytes at a time
            R.favor_ssm_scan(f.handle, u, u, A, bc, bc, None, None, None, st.data_ptr() + 4, None, B, None,
                             torch.empty_like(u), B, L)
        assert e.value.status == BAD
        off = A.data_ptr() + 2                      # parameters and tensors start on their elements
        for call in (lambda: R.favor_ssm_scan(f.handle, u, u, off, bc, bc, None, None, None, None, None, 0, None,
                                              torch.empty_like(u), B, L),
                     lambda: R.favor_conv_causal(f.handle, u, off, None, 1, None, None, 0, None, torch.empty_like(u), B, L),
                     lambda: R.favor_conv_causal(f.handle, u.data_ptr() + 1, w, None, 1, None, None, 0, None,
                                                 torch.empty_like(u), B, L, stream=0)):
            with pytest.raises(R.FavorError) as e:
                call()
            assert e.value.status == BAD and "aligned" in str(e.value)
        assert R.favor_launch_count() == n0


def _offline_ssm(monkeypatch, calls):
    """An Ssm of CPU tensors whose library only records the calls."""
    import torch
    from random_feature_gb300 import ssm

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    monkeypatch.setattr(ssm, "lib", Lib)
    f, cpu, f4 = object.__new__(R.Ssm), torch.device("cpu"), torch.float32
    f.D, f.N, f.G, f.K, f.handle, f.device, f._index, f._lib = 4, 8, 1, 2, None, cpu, 0, Lib()
    f._t, f._f32, f._i32, f._dims = f4, f4, torch.int32, (4,)
    f._weight, f._vec, f._A = ((4, 2), f4, cpu), ((4,), f4, cpu), ((4, 8), f4, cpu)
    return f


def test_pools_without_pages_are_refused(monkeypatch):
    """A pool of no pages has no address: it is refused, not taken for an absent one."""
    import torch
    calls = []
    f = _offline_ssm(monkeypatch, calls)
    x, bc, A, w = torch.zeros(2, 3, 4), torch.zeros(2, 3, 1, 8), torch.zeros(4, 8), torch.zeros(4, 2)
    x1, b1 = x[:, 0].contiguous(), bc[:, 0].contiguous()
    pages = torch.zeros(2, dtype=torch.int32)
    for kw in ({}, {"pages": pages}):
        for bad, name in ((lambda: f.conv(x, w, window=torch.zeros(0, 1, 4), **kw), "window"),
                          (lambda: f.conv_step(x1, w, torch.zeros(0, 1, 4), **kw), "window"),
                          (lambda: f.scan(x, x, A, bc, bc, state=torch.zeros(0, 4, 8), **kw), "state"),
                          (lambda: f.scan_step(x1, x1, A, b1, b1, torch.zeros(0, 4, 8), **kw), "state")):
            with pytest.raises(ValueError, match=name):
                bad()
    assert not calls
    f.conv(x, w, window=torch.zeros(2, 1, 4))
    f.scan(x, x, A, bc, bc, state=torch.zeros(2, 4, 8))
    assert [c[0] for c in calls] == ["favor_conv_causal", "favor_ssm_scan"]


def test_compaction_moves_pools_of_a_generator(monkeypatch):
    """The other pools may come from any iterable, one that can be walked once among them."""
    import torch
    from types import SimpleNamespace
    from random_feature_gb300 import ssm
    calls = []
    f = _offline_ssm(monkeypatch, calls)
    monkeypatch.setattr(ssm, "lib", lambda: f._lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    pool = lambda at: SimpleNamespace(numel=lambda: 8, dim=lambda: 2, is_cuda=True, is_contiguous=lambda: True,
                                      shape=(4, 2), element_size=lambda: 4, get_device=lambda: 0, data_ptr=lambda: at)
    table = torch.tensor([3, 1], dtype=torch.int32)
    monkeypatch.setattr(ssm, "_indices", lambda *a: None)
    R.pages_compact(pool(64), table, others=(pool(at) for at in (128, 256)))
    assert [c[0] for c in calls] == ["favor_pages_compact", "favor_pages_move", "favor_pages_move"]
    assert [c[1][0] for c in calls] == [64, 128, 256]
    calls.clear()
    bad = pool(256)
    bad.shape = (5, 2)
    with pytest.raises(ValueError, match=r"others\[1\]"):      # before anything is moved
        R.pages_compact(pool(64), table, others=(p for p in (pool(128), bad)))
    assert not calls


@pytest.mark.gpu
def test_compaction_of_a_generator_on_the_device():
    import torch
    pool = torch.arange(6, device="cuda", dtype=torch.float32).view(6, 1)
    wins = [pool * 10, pool * 100]
    table = torch.tensor([5, 2, 4], dtype=torch.int32, device="cuda")
    new, live = R.pages_compact(pool, table, others=(w for w in wins))
    assert new.tolist() == [1, 2, 0] and live.tolist() == [3]
    assert pool[:3, 0].tolist() == [4, 5, 2]
    for w, scale in zip(wins, (10, 100)):
        assert w[:3, 0].tolist() == [4 * scale, 5 * scale, 2 * scale]
