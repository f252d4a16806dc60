"""GPU tests of the page calls: copies and forks, clearing, compaction, against the oracle's rules;
results are copies of bytes, so they are equal."""
import numpy as np
import pytest
import torch

import oracle as O
import random_feature_gb300 as R

pytestmark = pytest.mark.gpu

# page shapes and types: 16-byte, 4-byte, 2-byte and 1-byte multiples, pages longer than a block's share
PAGES = [((4, 64), torch.float32), ((5,), torch.float32), ((3, 7), torch.bfloat16), ((13,), torch.uint8),
         ((257, 65), torch.float32), ((3, 1001), torch.bfloat16)]


def _pool(P, page, dtype, seed):
    r = np.random.default_rng(seed)
    return torch.from_numpy(r.integers(0, 120, (P, *page)).astype(np.uint8)).to("cuda", dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _np(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("page,dtype", PAGES, ids=[f"{'x'.join(map(str, p))}-{str(d)[6:]}" for p, d in PAGES])
def test_copy_and_fork(page, dtype):
    a, b = _pool(9, page, dtype, 1), _pool(6, page, dtype, 2)
    src, dst = [1, 1, 8, 9, -1, 0, 3, 2 ** 31 - 1], [0, 3, 3, 1, 2, 6, 5, 4]
    want, done = O.pages_copy(_np(b), _np(a), src, dst, same=False)
    got = R.pages_copy(b, a, _ints(src), _ints(dst))
    assert got.tolist() == done == [1, 1, 0, 0, 0, 0, 1, 0]
    assert np.array_equal(_np(b), want)
    # one pool: forks, a destination that the call reads, one named twice, a page onto itself
    src, dst = [1, 1, 4, 5, 7, 2], [0, 3, 5, 6, 7, 0]
    want, done = O.pages_copy(_np(a), _np(a), src, dst, same=True)
    got = R.pages_copy(a, a, _ints(src), _ints(dst))
    assert got.tolist() == done == [1, 1, 0, 1, 1, 0]
    assert np.array_equal(_np(a), want)


@pytest.mark.parametrize("page,dtype", PAGES, ids=[f"{'x'.join(map(str, p))}-{str(d)[6:]}" for p, d in PAGES])
def test_clear(page, dtype):
    a = _pool(7, page, dtype, 3) + 1
    want = _np(a)
    want[[2, 6]] = 0
    R.pages_clear(a, _ints([6, -1, 2, 7, 2]))
    assert np.array_equal(_np(a), want)


@pytest.mark.parametrize("P,S,seed", [(1, 1, 0), (5, 3, 1), (40, 25, 2), (64, 64, 3), (1000, 300, 4), (3001, 2000, 5)])
def test_compact(P, S, seed):
    r = np.random.default_rng(seed)
    table = r.integers(-2, P + 2, S).tolist()
    pool, win = _pool(P, (3, 8), torch.float32, seed), _pool(P, (5,), torch.bfloat16, seed + 1)
    want, new, live, where = O.pages_compact(_np(pool), table)
    wwin = O.pages_compact(_np(win), table)[0]
    got, n = R.pages_compact(pool, _ints(table), others=[win])
    assert got.tolist() == new and n.tolist() == [live]
    assert np.array_equal(_np(pool), want) and np.array_equal(_np(win), wwin)
    # again: nothing is left to move
    again, n = R.pages_compact(pool, got, others=[win])
    assert torch.equal(again, got) and n.tolist() == [live] and np.array_equal(_np(pool), want)


@pytest.mark.parametrize("table", [[-1, -1], [9, 3], [0, 1, 2], [11] * 5, list(range(11, -1, -1)), [6, 7, 8, 9, 10, 11]])
def test_compact_extremes(table):
    pool = _pool(12, (300,), torch.float32, 6)
    want, new, live, _ = O.pages_compact(_np(pool), table)
    got, n = R.pages_compact(pool, _ints(table))
    assert got.tolist() == new and n.tolist() == [live] and np.array_equal(_np(pool), want)


def test_compact_largest_table():
    """As many pages as the call takes."""
    P = 1 << 17
    r = np.random.default_rng(7)
    table = r.integers(0, P, 50000)
    pool = torch.arange(P, device="cuda", dtype=torch.int32)[:, None].contiguous()
    got, n = R.pages_compact(pool, _ints(table.tolist()))
    uniq = np.unique(table)
    U = len(uniq)
    assert n.item() == U
    # every entry's page holds what it held, pages below U are the live ones, those already there stayed
    now = got.cpu().numpy()
    host = pool.cpu().numpy()[:, 0]
    assert np.array_equal(host[now], table) and now.max() < U and np.array_equal(np.sort(host[:U]), uniq)
    assert np.array_equal(now[table < U], table[table < U])
    low = np.setdiff1d(np.arange(U), uniq)
    assert np.array_equal(host[low], uniq[uniq >= U])


def test_pages_of_a_serving_cache():
    """Favor states and scan states of a few sequences in pages: decode, fork a beam, free a sequence,
    compact, decode on; every sequence goes on as it does alone."""
    D, N, P = 48, 16, 10
    r = np.random.default_rng(8)
    f32 = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).cuda()
    A = -torch.exp(f32(D, N))
    w = f32(D, 4)
    with R.Ssm(D, N, 1, 4, "f32", P, 8, training=False) as f:
        def step(x, dt, Bm, Cm, win, state, pages=None):
            return f.scan_step(f.conv_step(x, w, win, pages=pages), dt, A, Bm, Cm, state, pages=pages)
        tok = lambda n: (f32(n, D), f32(n, D), f32(n, 1, N), f32(n, 1, N))
        win, state = f.new_window(P), f.new_state(P)
        slots = [7, 2, 9]
        alone = [(f.new_window(1), f.new_state(1)) for _ in slots]
        def both(slots, alone):
            t = tok(len(slots))
            got = step(*t, win, state, _ints(slots))
            want = torch.cat([step(*(a[i:i + 1] for a in t), *alone[i]) for i in range(len(slots))])
            assert torch.equal(got, want)
        for _ in range(3):
            both(slots, alone)
        # sequence 0 forks into page 4; sequence 1 is freed
        assert R.pages_copy(state, state, _ints([7]), _ints([4])).item() == 1
        assert R.pages_copy(win, win, _ints([7]), _ints([4])).item() == 1
        slots, alone = [7, 9, 4], [alone[0], alone[2], tuple(t.clone() for t in alone[0])]
        both(slots, alone)
        table, n = R.pages_compact(state, _ints(slots), others=[win])
        assert n.item() == 3 and sorted(table.tolist()) == [0, 1, 2]
        slots = table.tolist()
        for _ in range(2):
            both(slots, alone)
        # a new sequence on a page that held another one
        new = next(p for p in range(P) if p not in slots)
        R.pages_clear(state, _ints([new]))
        R.pages_clear(win, _ints([new]))
        both(slots + [new], alone + [(f.new_window(1), f.new_state(1))])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_of_favor_states(dtype):
    """States [H, m, dv+1] of the stateful FAVOR+ calls as pages: sequences are decoded, one is forked, one is
    freed, the live ones move together and are decoded on as the first pages of the pool; every sequence goes
    on as it does alone.  Odd pages (65 columns), and odd rows of them."""
    H, m, d, dv, P, T = 3, 32, 16, 64, 9, 5
    r = np.random.default_rng(9)
    omega = r.standard_normal((H, m, d)).astype(np.float32)
    t = lambda n, w: torch.from_numpy((0.5 * r.standard_normal((n, H, T, w))).astype(np.float32)).cuda() \
        .to(torch.float32 if dtype == "f32" else torch.bfloat16)
    with R.Favor(H, m, d, dv, "softmax_pos", dtype, omega, 0.5, P, 64) as f:
        pool = f.new_state(P)
        alone = [f.new_state(1) for _ in range(3)]

        def both(n):
            """T tokens of the first n pages, and of the same sequences alone."""
            q, k, v = t(n, d), t(n, d), t(n, dv)
            got = f.causal_step(q, k, v, pool[:n])
            want = torch.cat([f.causal_step(q[i:i + 1], k[i:i + 1], v[i:i + 1], alone[i]) for i in range(n)])
            assert torch.equal(got, want)
            assert torch.equal(pool[:n], torch.cat(alone))
        both(3)
        both(3)
        # sequence 2 forks into pages 8 and 5; sequence 0 ends
        assert R.pages_copy(pool, pool, _ints([2, 2]), _ints([8, 5])).tolist() == [1, 1]
        assert torch.equal(pool[8:9], alone[2]) and torch.equal(pool[5:6], alone[2])
        table, n = R.pages_compact(pool, _ints([1, 2, 8, 5]))
        assert n.item() == 4 and sorted(table.tolist()) == [0, 1, 2, 3]
        seqs = [alone[1], alone[2], alone[2].clone(), alone[2].clone()]
        alone = [None] * 4
        for at, s in zip(table.tolist(), seqs):
            alone[at] = s
        both(4)
        # a new sequence on a cleared page
        R.pages_clear(pool, _ints([4]))
        assert (pool[4] == 0).all()
        alone.append(f.new_state(1))
        both(5)
        # the states of prompts, added up by the stateful call, in pages as well
        k, v = t(1, d), t(1, dv)
        one = f.kv_state(k, v)
        assert R.pages_copy(pool, one, _ints([0]), _ints([7])).tolist() == [1] and torch.equal(pool[7:8], one)
        q = t(1, d)
        assert torch.equal(f.attn_from_state(q, pool[7:8]), f.attn_from_state(q, one))
