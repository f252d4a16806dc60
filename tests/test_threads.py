"""Two host threads that call one handle, both on one stream: the device runs the calls one after the
other, but a call is several launches on the handle's workspace, so these must not mix with another's."""
import threading

import pytest
import torch

import random_feature_gb300 as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pair", [("scan", "scan"), ("scan", "scan_backward"), ("scan_backward", "conv_backward"),
                                  ("conv_backward", "conv_backward")], ids="-".join)
def test_two_threads_on_one_handle(pair):
    B, L, D, N, K, turns = 1, 2048, 64, 16, 4, 300
    with R.Ssm(D, N, 1, K, "f32", B, L) as f:
        def worker(kind, seed):
            """(run(out), outputs of one call alone)."""
            g = torch.Generator(device="cuda").manual_seed(seed)
            rn = lambda *s: torch.randn(*s, device="cuda", generator=g)
            x, dt, do, Bm, Cm = rn(B, L, D), rn(B, L, D), rn(B, L, D), rn(B, L, 1, N), rn(B, L, 1, N)
            A, w = -torch.exp(rn(D, N)), rn(D, K)
            du, ddt, dB, dC = (torch.empty_like(t) for t in (x, x, Bm, Bm))

            def run(out):
                if kind == "scan":
                    R.favor_ssm_scan(f.handle, x, dt, A, Bm, Cm, None, None, None, None, None, 0, None, out, B, L,
                                     stream=0)
                elif kind == "scan_backward":
                    R.favor_ssm_scan_backward(f.handle, x, dt, A, Bm, Cm, None, None, None, None, do, du, ddt, out,
                                              dB, dC, None, None, None, B, L, stream=0)
                else:
                    R.favor_conv_causal_backward(f.handle, x, w, None, 1, None, do, du, out, None, B, L, stream=0)
            shape = {"scan": (B, L, D), "scan_backward": (D, N), "conv_backward": (D, K)}[kind]
            want = torch.empty(shape, device="cuda")
            run(want)
            return run, want, torch.empty(turns, *shape, device="cuda")

        workers = [worker(kind, 5 + i) for i, kind in enumerate(pair)]
        torch.cuda.synchronize()
        start, failed = threading.Barrier(2), []

        def go(run, outs):
            try:
                rows = list(outs)
                start.wait(30)
                for o in rows:
                    run(o)
            except Exception as e:
                failed.append(e)
        threads = [threading.Thread(target=go, args=(run, outs)) for run, _, outs in workers]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed
        for _, want, outs in workers:
            wrong = (outs != want).flatten(1).any(1).sum().item()
            assert wrong == 0, f"{wrong} of {turns} results differ"
