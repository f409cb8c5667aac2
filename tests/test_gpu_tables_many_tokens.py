"""GPU tests of tables for lists of more than 4,096 tokens, which take two launches, with everything that the second one
reads again and writes over updated in place: refusals, bad lengths and queues, steps in a captured graph, another stream.
Whole numbers: every output is equal."""
import numpy as np
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv
from test_gpu_tables import Host, check_lists, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("B,mb,NB,bs,T,seed", [(1, 800, 900, 16, 4097, 0), (40, 60, 1500, 16, 5000, 1), (500, 30, 4000, 8, 9000, 2),
                                               (3000, 6, 9000, 4, 20000, 3), (8192, 3, 20000, 16, 70000, 4)])
def test_steps_in_place(B, mb, NB, bs, T, seed):
    """Refused for blocks, for tokens and for rows that are full (of the 500 all are granted), sequences that bring
    nothing, blocks given back."""
    rng = np.random.default_rng(seed)
    h = Host(B, mb, NB, bs, free=rng.permutation(NB).tolist(), head=int(rng.integers(0, NB)))
    tables, lens, queue, state = h.device()
    out = pkv.make_step_tables(B, T)._replace(context_lens=lens, queue_state=state)
    refused = 0
    for step in range(8):
        new = np.where(rng.random(B) < 0.5, rng.integers(0, max(2, 3 * T // B), B), rng.integers(0, 2, B))
        before = list(h.lens)
        want = h.extend(new.tolist(), T)
        refused += sum(int(n > 0 and a == b) for n, a, b in zip(new, before, h.lens))
        got = pkv.extend_tables(tables, lens, dev(new), queue, state, bs, T, out=out)
        assert got.context_lens.data_ptr() == lens.data_ptr() and got.queue_state.data_ptr() == state.data_ptr()
        check_lists(got, *want)
        h.check(tables, lens, queue, state)
        done = (rng.random(B) < 0.4).astype(np.int32)
        h.release(done.tolist(), bs + 1, 3)
        pkv.release_tables(tables, lens, queue, state, bs, finished=dev(done), window=bs + 1, sinks=3)
        h.check(tables, lens, queue, state)
    assert refused > 0 or B == 500
    assert pkv.device_status() in ((0, 0), (7, pkv.FLAG_BAD_CONTEXT))  # (rows that are full refuse more)


@pytest.mark.parametrize("free", [0, 1, 4, 5, 6, 9, 10])
@pytest.mark.parametrize("T", [4097, 4100, 40000])
def test_who_is_refused(free, T):
    big = T - 40
    h = Host(7, T // 4 + 8, T, 4)
    for s, c in enumerate([3, 4, 5, 0, 7, 2, 0]):
        h.extend([c if i == s else 0 for i in range(7)], 100)
    h.free = h.free[:free + -(-big // 4)]
    tables, lens, queue, state = h.device()
    new = [1, 1, 2, 9, 1, 15, big]  # needs no block, one, none, three, none, four, many; the tokens fit up to the sixth or all
    out = pkv.make_step_tables(7, T)._replace(context_lens=lens, queue_state=state)
    want = h.extend(new, T)
    check_lists(pkv.extend_tables(tables, lens, dev(new), queue, state, 4, T, out=out), *want)
    h.check(tables, lens, queue, state)
    assert pkv.device_status() == (0, 0)


def test_bad_lengths_and_queues():
    T = 5000
    h = Host(5, 3, 20, 4)
    h.extend([4, 0, 12, 3, 0], 100)
    tables, lens, queue, state = h.device()
    lens[1] = -3
    out = pkv.make_step_tables(5, T)._replace(context_lens=lens, queue_state=state)
    want = h.extend([1, 0, 0, 0, 4], T)
    check_lists(pkv.extend_tables(tables, lens, dev([1, 2, 1, -5, 4]), queue, state, 4, T, out=out), *want)
    assert lens.cpu().tolist() == [5, -3, 12, 3, 4]
    assert pkv.device_status() == (7, pkv.FLAG_BAD_CONTEXT)
    for wrong in ([-1, 3], [20, 3], [0, 21], [0, -1]):
        state.copy_(dev(wrong))
        kept = tables.clone()
        o = pkv.extend_tables(tables, lens, dev([1, 0, 0, 1, 1]), queue, state, 4, T, out=out)
        # an empty queue: what fits the blocks that are there
        assert o.query_start.cpu().tolist()[0] == 0 and torch.equal(kept, tables)
        assert state.cpu().tolist() == [0, 0]
        flags = pkv.device_status()[1]
        assert flags & pkv.FLAG_BAD_QUEUE and not flags & ~(pkv.FLAG_BAD_QUEUE | pkv.FLAG_BAD_CONTEXT)


def test_captured_steps():
    """The same launches replayed: each step from where the one before left lengths and queue."""
    B, T, bs = 300, 6000, 16
    rng = np.random.default_rng(7)
    h = Host(B, 40, 9000, bs, head=8990)
    tables, lens, queue, state = h.device()
    new = dev(np.zeros(B))
    out = pkv.make_step_tables(B, T)._replace(context_lens=lens, queue_state=state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkv.extend_tables(tables, lens, new, queue, state, bs, T, out=out)  # nothing new: nothing changes
    torch.cuda.current_stream().wait_stream(side)
    h.check(tables, lens, queue, state)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.extend_tables(tables, lens, new, queue, state, bs, T, out=out)
    for _ in range(6):
        asked = rng.integers(0, 35, B)
        new.copy_(dev(asked))
        want = h.extend(asked.tolist(), T)
        g.replay()
        check_lists(out, *want)
        h.check(tables, lens, queue, state)
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        asked = rng.integers(0, 35, B)
        want = h.extend(asked.tolist(), T)
        got = pkv.extend_tables(tables, lens, dev(asked), queue, state, bs, T, out=out, stream=side)
        side.synchronize()
    check_lists(got, *want)
    h.check(tables, lens, queue, state)
    assert pkv.device_status() == (0, 0)
