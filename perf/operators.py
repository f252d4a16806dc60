"""The sequence-mixing operators beside FAVOR+ attention, as cases to be measured: the short causal
convolution and the selective state space scan (prompts, single tokens, gradients) and the pages of
a cache of recurrent states (copying and forking, compacting).

``run`` computes a case in elementary torch operations while ``own`` is false, and through the
library's calls where it is true.  ``exact`` is the operators' definition in float64.
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 64 sequences: the convolution's window pages are read and moved on
        dict(name="conv_step_64", op="conv_step", B=64, D=2048, K=4, dtype="bf16", P=96),
        # a batch of prompts through the convolution (the causal workload's 4 x 8192 tokens)
        dict(name="conv_prompt", op="conv", B=4, L=8192, D=1024, K=4, dtype="bf16", ragged=False),
        # the convolution's gradients in a training step (8 x 4096 tokens), fp32 storage
        dict(name="conv_train_f32", op="conv_bwd", B=8, L=4096, D=1536, K=4, dtype="f32", ragged=False),
        # one decoding step of one sequence: latency
        dict(name="scan_step_1", op="scan_step", B=1, D=2048, N=16, G=1, dtype="bf16", P=1),
        # one decoding step of a full serving batch, states in pages of a larger pool
        dict(name="scan_step_256", op="scan_step", B=256, D=2048, N=16, G=1, dtype="bf16", P=320),
        # a padded batch of prompts of very different lengths, odd width, fp32 storage
        dict(name="scan_ragged_f32", op="scan", B=3, L=1000, D=500, N=16, G=1, dtype="f32", ragged=True),
        # the encoder-sized batch: 8 x 4096 tokens
        dict(name="scan_prompt", op="scan", B=8, L=4096, D=1536, N=16, G=1, dtype="bf16", ragged=False),
        # one very long context: few channels, the work has to be split along the sequence
        dict(name="scan_long", op="scan", B=1, L=65536, D=1024, N=16, G=1, dtype="bf16", ragged=False),
        # the scan's gradients in a training step (4 x 8192 tokens)
        dict(name="scan_train", op="scan_bwd", B=4, L=8192, D=1024, N=16, G=1, dtype="bf16", ragged=False),
        # the same with odd sizes, several groups of B and C, fp32 storage
        dict(name="scan_train_f32", op="scan_bwd", B=2, L=777, D=500, N=32, G=4, dtype="f32", ragged=True),
        # beams forked from one another: pages that hold a FAVOR+ state [12, 256, 65]
        dict(name="pages_fork", op="pages_copy", P=128, E=12 * 256 * 65, n=48),
        # half of a pool of scan states has been freed: the live pages move together
        dict(name="pages_compact", op="pages_compact", P=1024, E=2048 * 16, S=600),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_bwd", "conv_step", "scan", "scan", "scan_bwd", "scan_bwd", "scan_step",
                     "scan_step", "pages_copy", "pages_compact"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "pages_copy":
        P = _log_int(rng, 8, 256)
        return dict(op=op, P=P, E=4 * _log_int(rng, 64, 50000), n=_log_int(rng, 1, max(1, P // 2)))
    if op == "pages_compact":
        P = _log_int(rng, 8, 1024)
        return dict(op=op, P=P, E=4 * _log_int(rng, 64, 8192), S=_log_int(rng, 1, P))
    D = _log_int(rng, 64, 2048)
    if rng.random() < 0.6:
        D = max(64, D // 64 * 64)
    if op in ("conv_step", "scan_step"):
        B = _log_int(rng, 1, 256)
        case = dict(op=op, B=B, D=D, dtype=dtype, P=B + rng.randrange(0, 64))
    else:
        B = _log_int(rng, 1, 8)
        most = (1 << 25) if op == "scan_bwd" else (1 << 26)
        L = _log_int(rng, 1, min(8192 if op == "scan_bwd" else 16384, most // (B * D)))
        case = dict(op=op, B=B, L=L, D=D, dtype=dtype, ragged=rng.random() < 0.4)
    if op.startswith("conv"):
        case["K"] = rng.choice([2, 3, 4])
    else:
        N = rng.choice([8, 16, 16, 16, 32, 64])
        if B * D * case.get("L", 1) * N > (1 << 30 if op != "scan_bwd" else 1 << 29):
            N = 16
        case["N"] = N
        case["G"] = rng.choice([g for g in (1, 1, 1, 2, 4) if D % g == 0])
    return case


def _lens(case):
    """Lengths of a ragged batch, from its sizes: the first row is full, others run from 0 to L."""
    B, L = case["B"], case["L"]
    r = random.Random(7919 * B + L)
    return [L] + [r.choice([0, 1, r.randint(0, L), r.randint(0, L)]) for _ in range(B - 1)]


def _tokens(case):
    if "L" not in case:
        return case["B"]
    return sum(_lens(case)) if case["ragged"] else case["B"] * case["L"]


def work(case):
    op = case["op"]
    if op == "pages_copy":
        return dict(bytes=2 * 4 * case["n"] * case["E"], flops=0)
    if op == "pages_compact":
        moved = len(_moves(_live(case)))
        return dict(bytes=2 * 4 * moved * case["E"], flops=0)
    s = 4 if case["dtype"] == "f32" else 2
    T, D = _tokens(case), case["D"]
    if op.startswith("conv"):
        K = case["K"]
        if op == "conv_step":
            return dict(bytes=T * D * s * (2 + 2 * (K - 1)) + D * (K + 1) * 4, flops=T * D * (2 * K + 5))
        if op == "conv":
            return dict(bytes=T * D * s * 2 + case["B"] * D * s * 2 * (K - 1) + D * (K + 1) * 4,
                        flops=T * D * (2 * K + 5))
        return dict(bytes=T * D * s * 3 + D * (K + 1) * 8, flops=T * D * (6 * K + 12))
    N, G = case["N"], case["G"]
    par = D * N * 4 + D * 8
    if op == "scan_step":
        return dict(bytes=T * D * s * 4 + T * G * N * s * 2 + T * D * N * 8 + par, flops=T * D * (7 * N + 14))
    if op == "scan":
        return dict(bytes=T * D * s * 4 + T * G * N * s * 2 + case["B"] * D * N * 8 + par,
                    flops=T * D * (7 * N + 14))
    return dict(bytes=T * D * s * 7 + T * G * N * s * 4 + 2 * par, flops=T * D * (21 * N + 40))


# ---------------------------------------------------------------- inputs
def _live(case):
    """Pages named by the table's entries (-1: a free entry); some pages are shared by two entries."""
    r = random.Random(31 * case["P"] + case["S"])
    pages = r.sample(range(case["P"]), case["S"])
    out = []
    for i, p in enumerate(pages):
        x = r.random()
        out.append(-1 if x < 0.1 else out[r.randrange(i)] if x < 0.2 and i else p)
    return out


def _moves(table):
    live = sorted({p for p in table if p >= 0})
    n = len(live)
    return [p for p in live if p >= n]


def _inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=dev, dtype=torch.float32)

    op = case["op"]
    st = {}
    r = random.Random(seed)
    if op == "pages_copy":
        st["pool"] = randn(case["P"], case["E"])
        order = r.sample(range(case["P"]), case["P"])
        dst = order[:case["n"]]
        src = [r.choice(order[case["n"]:]) for _ in dst]
        st["src"] = torch.tensor(src, dtype=torch.int32, device=dev)
        st["dst"] = torch.tensor(dst, dtype=torch.int32, device=dev)
        return st
    if op == "pages_compact":
        st["pool"] = randn(case["P"], case["E"])
        st["table"] = torch.tensor(_live(case), dtype=torch.int32, device=dev)
        return st
    t = _DT[case["dtype"]]
    B, D = case["B"], case["D"]
    lead = (B, case["L"]) if "L" in case else (B,)
    if "L" in case and case["ragged"]:
        st["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
    if op.startswith("conv"):
        K = case["K"]
        st["x"] = randn(*lead, D).to(t)
        st["weight"] = randn(D, K) / math.sqrt(K)
        st["bias"] = 0.1 * randn(D)
        if op == "conv_bwd":
            st["dout"] = randn(*lead, D).to(t)
        else:
            P = case.get("P", B)
            st["window"] = randn(P, K - 1, D).to(t)
            if op == "conv_step":
                st["pages"] = torch.tensor(r.sample(range(P), B), dtype=torch.int32, device=dev)
        return st
    N, G = case["N"], case["G"]
    x = randn(*lead, D)
    st["u"] = (x * torch.sigmoid(x)).to(t)                       # what the convolution's activation gives
    st["dt"] = (0.5 * randn(*lead, D)).to(t)
    step = torch.exp(rand(D) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    st["dt_bias"] = step + torch.log(-torch.expm1(-step))        # softplus(dt_bias) spread over 0.001 .. 0.1
    st["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(0.1 * randn(D, N))
    st["Bm"] = randn(*lead, G, N).to(t)
    st["Cm"] = randn(*lead, G, N).to(t)
    st["skip"] = 1 + 0.1 * randn(D)
    st["z"] = randn(*lead, D).to(t)
    if op == "scan_bwd":
        st["dout"] = randn(*lead, D).to(t)
    else:
        P = case.get("P", B)
        st["state"] = 0.3 * randn(P, D, N)
        if op == "scan_step":
            st["pages"] = torch.tensor(r.sample(range(P), B), dtype=torch.int32, device=dev)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["op"] = case["op"]
    if own and not case["op"].startswith("pages"):
        import random_feature_gb300 as R
        st["ssm"] = R.Ssm(case["D"], case.get("N", 16), case.get("G", 1), case.get("K", 4), case["dtype"],
                          case["B"], case.get("L", 1))
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    return (_own if own else _plain)[st["op"]](st)


def _own_conv(s):
    out = s["ssm"].conv(s["x"], s["weight"], s["bias"], window=s["window"], lens=s.get("lens"))
    return out, s["window"]


def _own_conv_step(s):
    return s["ssm"].conv_step(s["x"], s["weight"], s["window"], s["bias"], pages=s["pages"]), s["window"]


def _own_conv_bwd(s):
    return s["ssm"].conv_backward(s["x"], s["weight"], s["dout"], s["bias"], lens=s.get("lens"))


def _own_scan(s):
    out = s["ssm"].scan(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"],
                        state=s["state"], lens=s.get("lens"))
    return out, s["state"]


def _own_scan_step(s):
    out = s["ssm"].scan_step(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], skip=s["skip"], z=s["z"],
                             dt_bias=s["dt_bias"], pages=s["pages"])
    return out, s["state"]


def _own_scan_bwd(s):
    return s["ssm"].scan_backward(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dout"], skip=s["skip"], z=s["z"],
                                  dt_bias=s["dt_bias"], lens=s.get("lens"))


def _own_pages_copy(s):
    import random_feature_gb300 as R
    return R.pages_copy(s["pool"], s["pool"], s["src"], s["dst"]), s["pool"]


def _own_pages_compact(s):
    import random_feature_gb300 as R
    table, live = R.pages_compact(s["pool"], s["table"])
    return table, live, s["pool"]


_own = dict(conv=_own_conv, conv_step=_own_conv_step, conv_bwd=_own_conv_bwd, scan=_own_scan,
            scan_step=_own_scan_step, scan_bwd=_own_scan_bwd, pages_copy=_own_pages_copy,
            pages_compact=_own_pages_compact)


# The plain forms: fp32 elementary operations, rounded once at the end.
def _valid(s, lead):
    """[B, L, 1] truth values of the rows inside each sequence, or None."""
    if "lens" not in s:
        return None
    return (torch.arange(lead[1], device="cuda")[None, :] < s["lens"][:, None])[..., None]


def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _taps(xp, w, bias, L):
    p = bias + w[:, 0] * xp[:, 0:L]
    for k in range(1, w.shape[1]):
        p = p + w[:, k] * xp[:, k:k + L]
    return p


def _plain_conv(s):
    x, w = s["x"], s["weight"]
    K = w.shape[1]
    B, L, D = x.shape
    xp = torch.cat([s["window"], x], 1)
    out = _silu(_taps(xp.float(), w, s["bias"], L)).to(x.dtype)
    ok = _valid(s, x.shape)
    if ok is None:
        s["window"].copy_(xp[:, L:])
    else:
        out = torch.where(ok, out, torch.zeros_like(out))
        idx = s["lens"].long()[:, None] + torch.arange(K - 1, device=x.device)
        s["window"].copy_(torch.gather(xp, 1, idx[..., None].expand(B, K - 1, D)))
    return out, s["window"]


def _plain_conv_step(s):
    x, w, pages = s["x"], s["weight"], s["pages"].long()
    xp = torch.cat([s["window"][pages], x[:, None]], 1)
    out = _silu(_taps(xp.float(), w, s["bias"], 1))[:, 0].to(x.dtype)
    s["window"][pages] = xp[:, 1:]
    return out, s["window"]


def _plain_conv_bwd(s):
    x, w, g = s["x"].float(), s["weight"], s["dout"].float()
    K = w.shape[1]
    B, L, D = x.shape
    ok = _valid(s, x.shape)
    if ok is not None:
        x = torch.where(ok, x, torch.zeros_like(x))
        g = torch.where(ok, g, torch.zeros_like(g))
    xp = torch.cat([x.new_zeros(B, K - 1, D), x], 1)
    p = _taps(xp, w, s["bias"], L)
    e = 1 / (1 + torch.exp(-p))
    g = g * (e * (1 + p * (1 - e)))
    gp = torch.cat([g, g.new_zeros(B, K - 1, D)], 1)
    dx = w[:, K - 1] * gp[:, 0:L]
    for k in range(K - 1):
        dx = dx + w[:, k] * gp[:, K - 1 - k:K - 1 - k + L]
    if ok is not None:
        dx = torch.where(ok, dx, torch.zeros_like(dx))
    dw = torch.stack([(g * xp[:, k:k + L]).sum((0, 1), dtype=torch.float64) for k in range(K)], -1)
    return dx.to(s["x"].dtype), dw.float(), g.sum((0, 1), dtype=torch.float64).float()


_BLOCK = 64


def _scan_block(s, t0, t1, dt, u, ok):
    """exp(dt A) and dt u B of tokens t0 .. t1-1, token first: [T, B, D, N]; a row behind its
    sequence's end leaves the state as it is."""
    D = u.shape[2]
    A = s["A"]
    Bm = s["Bm"][:, t0:t1].float().transpose(0, 1)
    Bm = Bm.repeat_interleave(D // Bm.shape[2], 2)                # [T, B, D, N]
    d = dt[:, t0:t1].transpose(0, 1)[..., None]
    a = torch.exp(d * A)
    b = d * u[:, t0:t1].transpose(0, 1)[..., None] * Bm
    if ok is not None:
        m = ok[:, t0:t1].transpose(0, 1)[..., None]
        a = torch.where(m, a, torch.ones_like(a))
        b = torch.where(m, b, torch.zeros_like(b))
    return a, b, Bm


def _plain_scan(s):
    u, z = s["u"].float(), s["z"].float()
    B, L, D = u.shape
    ok = _valid(s, u.shape)
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    h = s["state"].clone()
    y = torch.empty_like(u)
    for t0 in range(0, L, _BLOCK):
        t1 = min(L, t0 + _BLOCK)
        a, b, _ = _scan_block(s, t0, t1, dt, u, ok)
        for t in range(t1 - t0):
            h = torch.addcmul(b[t], a[t], h, out=b[t])
        Cm = s["Cm"][:, t0:t1].float().transpose(0, 1)
        Cm = Cm.repeat_interleave(D // Cm.shape[2], 2)
        y[:, t0:t1] = (b * Cm).sum(-1).transpose(0, 1)
    s["state"].copy_(h)
    out = ((y + s["skip"] * u) * _silu(z)).to(s["u"].dtype)
    if ok is not None:
        out = torch.where(ok, out, torch.zeros_like(out))
    return out, s["state"]


def _plain_scan_step(s):
    u, z, pages = s["u"].float(), s["z"].float(), s["pages"].long()
    D = u.shape[1]
    dt = _softplus(s["dt"].float() + s["dt_bias"])[..., None]
    Bm = s["Bm"].float()
    Bm = Bm.repeat_interleave(D // Bm.shape[1], 1)
    Cm = s["Cm"].float()
    Cm = Cm.repeat_interleave(D // Cm.shape[1], 1)
    h = torch.exp(dt * s["A"]) * s["state"][pages] + dt * u[..., None] * Bm
    s["state"][pages] = h
    y = (h * Cm).sum(-1) + s["skip"] * u
    return (y * _silu(z)).to(s["u"].dtype), s["state"]


def _plain_scan_bwd(s):
    dtype = s["u"].dtype
    u, z, do = s["u"].float(), s["z"].float(), s["dout"].float()
    B, L, D = u.shape
    A, G = s["A"], s["Bm"].shape[2]
    N = A.shape[1]
    ok = _valid(s, u.shape)
    if ok is not None:
        u, z, do = (torch.where(ok, t, torch.zeros_like(t)) for t in (u, z, do))
    raw = s["dt"].float() + s["dt_bias"]
    dt = _softplus(raw)
    e = 1 / (1 + torch.exp(-z))
    g = do * z * e                                                # gradient of y
    # forward: every state
    hs = u.new_empty(L + 1, B, D, N)
    hs[0] = 0
    y = torch.empty_like(u)
    for t0 in range(0, L, _BLOCK):
        t1 = min(L, t0 + _BLOCK)
        a, b, _ = _scan_block(s, t0, t1, dt, u, ok)
        for t in range(t1 - t0):
            torch.addcmul(b[t], a[t], hs[t0 + t], out=hs[t0 + t + 1])
        Cm = s["Cm"][:, t0:t1].float().transpose(0, 1).repeat_interleave(D // G, 2)
        y[:, t0:t1] = (hs[t0 + 1:t1 + 1] * Cm).sum(-1).transpose(0, 1)
    y = y + s["skip"] * u
    dz = do * y * (e * (1 + z * (1 - e)))
    dskip = (g * u).sum((0, 1), dtype=torch.float64)
    # backward
    du, ddt = s["skip"] * g, torch.empty_like(u)
    dB, dC = u.new_empty(L, B, G, N), u.new_empty(L, B, G, N)
    dA = A.new_zeros(A.shape, dtype=torch.float64)
    lam = u.new_zeros(B, D, N)                                    # a[t+1] lam[t+1]
    for t0 in reversed(range(0, L, _BLOCK)):
        t1 = min(L, t0 + _BLOCK)
        a, _, Bm = _scan_block(s, t0, t1, dt, u, ok)
        gt = g[:, t0:t1].transpose(0, 1)[..., None]
        lams = gt * s["Cm"][:, t0:t1].float().transpose(0, 1).repeat_interleave(D // G, 2)
        dC[t0:t1] = (gt * hs[t0 + 1:t1 + 1]).view(t1 - t0, B, G, D // G, N).sum(3)
        for t in reversed(range(t1 - t0)):
            lams[t] += lam
            lam = a[t] * lams[t]
        ut, dtt = u[:, t0:t1].transpose(0, 1)[..., None], dt[:, t0:t1].transpose(0, 1)[..., None]
        dB[t0:t1] = (lams * (dtt * ut)).view(t1 - t0, B, G, D // G, N).sum(3)
        lb = (lams * Bm).sum(-1).transpose(0, 1)
        q = lams * a * hs[t0:t1]
        if ok is not None:
            q = torch.where(ok[:, t0:t1].transpose(0, 1)[..., None], q, torch.zeros_like(q))
        du[:, t0:t1] += dt[:, t0:t1] * lb
        ddt[:, t0:t1] = u[:, t0:t1] * lb + (q * A).sum(-1).transpose(0, 1)
        dA += (q * dtt).sum((0, 1), dtype=torch.float64)
    draw_ = ddt / (1 + torch.exp(-raw))
    dB, dC = dB.transpose(0, 1), dC.transpose(0, 1)
    if ok is not None:
        du, draw_, dz = (torch.where(ok, t, torch.zeros_like(t)) for t in (du, draw_, dz))
        dB, dC = (torch.where(ok[..., None], t, torch.zeros_like(t)) for t in (dB, dC))
    return dict(du=du.to(dtype), ddt=draw_.to(dtype), dA=dA.float(), dB=dB.to(dtype).contiguous(),
                dC=dC.to(dtype).contiguous(), dskip=dskip.float(), dz=dz.to(dtype),
                ddt_bias=draw_.sum((0, 1), dtype=torch.float64).float())


def _plain_pages_copy(s):
    s["pool"][s["dst"].long()] = s["pool"][s["src"].long()]
    return torch.ones_like(s["src"]), s["pool"]


def _plain_pages_compact(s):
    pool, table = s["pool"], s["table"].long()
    P = pool.shape[0]
    live = torch.zeros(P + 1, dtype=torch.int64, device=pool.device)
    live[torch.where(table >= 0, table, P)] = 1
    live = live[:P]
    n = live.sum()
    at = torch.arange(P, device=pool.device)
    high, free = live * (at >= n), (1 - live) * (at < n)          # pages to move, pages to fill
    src, dst = torch.nonzero(high)[:, 0], torch.nonzero(free)[:, 0]
    pool[dst] = pool[src]
    where = at.clone()
    where[src] = dst
    new = torch.where(table >= 0, where[table.clamp(min=0)], -1)
    return new.int(), n.int().reshape(1), pool


_plain = dict(conv=_plain_conv, conv_step=_plain_conv_step, conv_bwd=_plain_conv_bwd, scan=_plain_scan,
              scan_step=_plain_scan_step, scan_bwd=_plain_scan_bwd, pages_copy=_plain_pages_copy,
              pages_compact=_plain_pages_compact)


# ---------------------------------------------------------------- definition in 64 bits
def exact(case, seed):
    """What run returns, in float64, token by token from the definition; gradients by reverse-mode
    differentiation of it.  Copies of pages are not computed: None."""
    op = case["op"]
    if op == "pages_copy":
        return None
    if op == "pages_compact":
        return None
    s = _inputs(case, seed)
    f = {k: v.double() for k, v in s.items() if v.is_floating_point()}
    lens = s["lens"].tolist() if "lens" in s else [case.get("L", 1)] * case["B"]
    if op.startswith("conv"):
        return _exact_conv(op, f, s, lens)
    return _exact_scan(op, f, s, lens)


def _exact_conv_row(x, past, w, bias):
    """One sequence x [T, D] after the inputs past [K-1, D]: silu of the depthwise correlation."""
    seq = torch.cat([past, x], 0)
    win = seq.unfold(0, w.shape[1], 1)                            # [T, D, K]
    p = torch.einsum("tdk,dk->td", win, w) + bias
    return p * torch.sigmoid(p), seq[x.shape[0]:]


def _exact_conv(op, f, s, lens):
    w, bias, x = f["weight"], f["bias"], f["x"]
    K, D = w.shape[1], w.shape[0]
    if op == "conv_step":
        out, win = torch.empty_like(x), f["window"]
        for b, p in enumerate(s["pages"].tolist()):
            o, win[p] = _exact_conv_row(x[b:b + 1], win[p].clone(), w, bias)
            out[b] = o[0]
        return out, win
    if op == "conv":
        out, win = torch.zeros_like(x), f["window"]
        for b, n in enumerate(lens):
            if n:
                out[b, :n], win[b] = _exact_conv_row(x[b, :n], win[b].clone(), w, bias)
        return out, win
    x, w, bias = (t.requires_grad_() for t in (x, w, bias))
    dx, dw, db = torch.zeros_like(x), torch.zeros_like(w), torch.zeros_like(bias)
    for b, n in enumerate(lens):
        if n:
            o, _ = _exact_conv_row(x[b, :n], x.new_zeros(K - 1, D), w, bias)
            gx, gw, gb = torch.autograd.grad(o, (x, w, bias), f["dout"][b, :n])
            dx += gx
            dw += gw
            db += gb
    return dx.detach(), dw.detach(), db.detach()


def _exact_scan(op, f, s, lens):
    if op == "scan_step":
        pages = s["pages"].long()
        state = f["state"]
        tok = {k: f[k][:, None] for k in ("u", "dt", "Bm", "Cm", "z")}
        out, h = _exact_tokens(tok, f, state[pages], [1] * len(lens))
        state[pages] = h
        return out[:, 0], state
    if op == "scan":
        return _exact_tokens(f, f, f["state"], lens)
    names = ("u", "dt", "A", "Bm", "Cm", "skip", "z", "dt_bias")
    ins = [f[k].requires_grad_() for k in names]
    h0 = f["u"].new_zeros(f["u"].shape[0], *f["A"].shape)
    out, _ = _exact_tokens(f, f, h0, lens)
    gr = torch.autograd.grad(out, ins, f["dout"])
    return dict(zip(("du", "ddt", "dA", "dB", "dC", "dskip", "dz", "ddt_bias"), gr))


def _exact_tokens(t, p, h, lens):
    """The recurrence over the tokens of t from the states h; rows behind a sequence's end give zeros."""
    Bn, L, D = t["u"].shape
    rep = D // t["Bm"].shape[2]
    n = torch.tensor(lens, device=h.device)
    full = min(lens) == L
    ys = []
    for i in range(L):
        step = torch.nn.functional.softplus(t["dt"][:, i] + p["dt_bias"], threshold=700.0).unsqueeze(-1)
        bi = t["Bm"][:, i].repeat_interleave(rep, 1)
        ci = t["Cm"][:, i].repeat_interleave(rep, 1)
        new = (step * p["A"]).exp() * h + step * bi * t["u"][:, i].unsqueeze(-1)
        h = new if full else torch.where((i < n)[:, None, None], new, h)
        ys.append(torch.einsum("bdn,bdn->bd", new, ci))
    y = torch.stack(ys, 1) + p["skip"] * t["u"]
    out = y * t["z"] * torch.sigmoid(t["z"])
    if not full:
        out = torch.where((torch.arange(L, device=h.device)[None, :] < n[:, None])[..., None], out,
                          torch.zeros_like(out))
    return out, h
