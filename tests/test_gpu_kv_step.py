"""Pages and slots of a step against the request-by-request restatement: every output is a whole number
and has to be equal."""
import numpy as np
import pytest

import oracle.step_ref as R
from parity_util import dev, host
from synth import rng

pytestmark = pytest.mark.gpu

S = pytest.importorskip("sparsity_amd")

I = np.int32


def _state(g, B, page, per, most, ended=0.0, begin=0.3, spare=3, short=None):
    """Requests that hold pages of a shuffled pool; the rest of the pool is on the stack."""
    fresh = g.integers(0, most + 1, B).astype(I)
    cached = g.integers(0, max(1, per * page - most + 1), B).astype(I)
    cached[g.random(B) < begin] = 0
    fresh[g.random(B) < ended] = -1
    pool = g.permutation(B * per + spare).astype(I)
    blocks = np.full((B, per), -7, I)
    n = 0
    for b in range(B):
        k = -(-int(cached[b]) // page)
        blocks[b, :k] = pool[n:n + k]
        n += k
    free = np.full(len(pool), -9, I)
    free[:len(pool) - n] = pool[n:]
    count = len(pool) - n if short is None else min(short, len(pool) - n)
    return cached, fresh, blocks, free, count


def _check(cached, fresh, blocks, free, count, page, T, in_place=False, slot=True):
    import torch
    B = len(cached)
    d = [dev(x) for x in (cached, fresh, blocks, free, np.array([count], I))]
    out = None
    if in_place or not slot:
        e = lambda n, t=torch.int32: torch.full((n,), 77, dtype=t, device="cuda")  # noqa: E731
        out = S.KvStep(e(T), e(T), e(T, torch.int64) if slot else None, d[0] if in_place else e(B), e(B + 1),
                       d[4] if in_place else e(1))
    print(B, page, blocks.shape, T, count, in_place, flush=True)
    r = S.kv_step(*d, page, T, out=out)
    rb, rf = blocks.copy(), free.copy()
    seq, pos, slots, lens, starts, left = R.kv_step(cached, fresh, rb, rf, count, page, T)
    assert np.array_equal(host(r.seq), seq) and np.array_equal(host(r.pos), pos)
    if slot:
        assert np.array_equal(host(r.slot), slots)
    assert np.array_equal(host(r.lens), lens) and np.array_equal(host(r.starts), starts)
    assert int(host(r.count)[0]) == left
    assert np.array_equal(host(d[2]), rb) and np.array_equal(host(d[3]), rf)
    if not in_place:
        assert np.array_equal(host(d[0]), cached) and int(host(d[4])[0]) == count
    assert np.array_equal(host(d[1]), fresh)
    return lens, starts


@pytest.mark.parametrize("B,page,per,most,T", [
    (1, 16, 4, 1, 1), (3, 1, 9, 4, 20), (64, 16, 8, 1, 64), (65, 7, 5, 30, 1500), (1000, 16, 6, 3, 2000),
    (1024, 8, 4, 2, 1100), (1025, 8, 4, 2, 2050), (2500, 24, 3, 6, 4096), (40, 64, 30, 700, 20000),
    (1500, 5, 9, 20, 16385), (9000, 3, 2, 2, 9001)])
@pytest.mark.parametrize("in_place", [False, True])
def test_steps(B, page, per, most, T, in_place):
    g = rng(B * 7 + T)
    _check(*_state(g, B, page, per, most, ended=0.2), page, T, in_place)


@pytest.mark.parametrize("B,page,per,most,T,short", [
    (10, 4, 6, 9, 100, 0), (10, 4, 6, 9, 100, 5), (300, 4, 6, 9, 5000, 100), (1300, 4, 3, 5, 6000, 700), (1300, 4, 6, 9, 9000, 700),
    (200, 8, 8, 40, 1000, None), (50, 1, 8, 8, 10, None)])
def test_pages_or_rows_that_do_not_suffice(B, page, per, most, T, short):
    """Pages run out, or the token rows do; requests that need no new page are still served."""
    lens, starts = _check(*_state(rng(B + T), B, page, per, most, ended=0.05, short=short), page, T)
    assert starts[-1] <= T


def test_a_table_row_that_is_full():
    cached, fresh = np.array([8, 7, 8, 3, 9], I), np.array([0, 1, 1, 2, 0], I)
    blocks = np.arange(10, dtype=I).reshape(5, 2)
    free = np.arange(20, 30, dtype=I)
    lens, starts = _check(cached, fresh, blocks, free, 10, 4, 16)     # rows of two pages of four tokens
    assert lens.tolist() == [8, 8, 8, 5, 9] and starts.tolist() == [0, 0, 1, 1, 3, 3]


def test_pages_of_ended_requests_serve_the_same_step():
    """An empty stack: the first request can only grow on what the others give back, its top first."""
    cached, fresh = np.array([4, 6, 8], I), np.array([5, -1, -1], I)
    blocks = np.array([[0, 90, 91], [1, 2, 92], [3, 4, 93]], I)
    free = np.zeros(6, I)
    lens, _ = _check(cached, fresh, blocks, free, 0, 4, 8)
    assert lens.tolist() == [9, 0, 0]


@pytest.mark.parametrize("count,cap", [(5, 6), (6, 6), (9, 6), (-3, 6), (0, 0)])
def test_a_stack_that_is_full_drops_pages(count, cap):
    cached, fresh = np.array([9, 5, 3], I), np.array([-1, -1, 0], I)
    blocks = np.arange(9, dtype=I).reshape(3, 3)
    _check(cached, fresh, blocks, np.full(cap, 50, I), count, 4, 3)


def test_lengths_at_the_ends_of_their_range():
    cached = np.array([-5, 2 ** 31 - 1, 2 ** 31 - 2, 0, -2 ** 31], I)
    fresh = np.array([2, 0, 3, 2 ** 31 - 1, -2 ** 31], I)
    blocks = np.arange(10, dtype=I).reshape(5, 2)
    _check(cached, fresh, blocks, np.arange(10, 16, dtype=I), 6, 2 ** 30, 4)
    _check(cached, fresh, blocks, np.arange(10, 16, dtype=I), 6, 4, 4)


def test_no_requests_and_no_rows():
    none = np.zeros(0, I)
    _check(none, none, np.zeros((0, 4), I), np.arange(3, dtype=I), 3, 16, 5)
    _check(none, none, np.zeros((0, 4), I), np.arange(3, dtype=I), 3, 16, 5000)
    _check(np.array([3, 4], I), np.array([0, -1], I), np.array([[1], [2]], I), np.zeros(2, I), 0, 4, 0)


def test_large_page_numbers():
    """Slots past 32 bits."""
    blocks = np.array([[2 ** 31 - 1, 2 ** 30]], I)
    _check(np.array([30], I), np.array([4], I), blocks, np.array([2 ** 31 - 3], I), 1, 32, 6)


def test_steps_without_slots():
    _check(*_state(rng(5), 33, 4, 6, 5, ended=0.1), 4, 100, slot=False)
    _check(*_state(rng(6), 33, 4, 60, 200, ended=0.1), 4, 5000, slot=False)
    _check(*_state(rng(7), 33, 4, 60, 200, ended=0.1), 4, 9000, slot=False)


@pytest.mark.parametrize("T", [40, 5000, 9000])
def test_steps_in_a_row_as_a_graph(T):
    """A captured step in place, replayed: lengths, tables and the stack move on as in eager steps."""
    import torch
    g = rng(11)
    B, page, per = 24, 4, 12
    cached, fresh, blocks, free, count = _state(g, B, page, per, 1, begin=1.0)
    d = [dev(x) for x in (cached, fresh, blocks, free, np.array([count], I))]
    e = lambda n, t=torch.int32: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
    out = S.KvStep(e(T), e(T), e(T, torch.int64), d[0], e(B + 1), d[4])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        S.kv_step(*d, page, T, out=out)
    for step in range(12):
        fresh = g.integers(-1 if step % 4 == 3 else 0, 6, B).astype(I)
        d[1].copy_(dev(fresh))
        graph.replay()
        seq, pos, slot, cached, _, count = R.kv_step(cached, fresh, blocks, free, count, page, T)
        for got, want in zip((out.seq, out.pos, out.slot, d[0], d[2], d[3]), (seq, pos, slot, cached, blocks, free)):
            assert np.array_equal(host(got), want), step
        assert int(host(d[4])[0]) == count
        held = np.concatenate([blocks[b, :-(-int(n) // page)] for b, n in enumerate(cached)] + [free[:count]])
        assert sorted(held) == list(range(B * per + 3))        # no page lost, none held twice
