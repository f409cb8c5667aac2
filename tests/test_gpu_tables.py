"""GPU tests of the tables built on the device (extend_tables, release_tables) against lists and a queue on the host,
and against the host allocator.  Whole numbers: every output is equal."""
import numpy as np
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dev(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


class Host:
    """Sequences' tables as lists and the free blocks as a queue."""

    def __init__(self, B, mb, NB, bs, free=None, head=0):
        self.B, self.mb, self.NB, self.bs = B, mb, NB, bs
        self.free = list(range(NB)) if free is None else list(free)
        self.lens = [0] * B
        self.rows = [[-1] * mb for _ in range(B)]
        self.head = head

    def device(self):
        queue = np.full(self.NB, -1)
        queue[(self.head + np.arange(len(self.free))) % self.NB] = self.free
        return dev(self.rows).view(self.B, self.mb), dev(self.lens), dev(queue), dev([self.head, len(self.free)])

    def extend(self, new, T):
        bs, want, brought, free = self.bs, 0, 0, len(self.free)
        start, slots, pos, seqs = [0], [], [], []
        for s, n in enumerate(new):
            c = self.lens[s]
            ok = n >= 0 and c + n <= self.mb * bs
            if ok:
                need = -(-(c + n) // bs) - -(-c // bs)
                want += need
                brought += n
                ok = (need == 0 or want <= free) and brought <= T
            if ok:
                for e in range(-(-c // bs), -(-(c + n) // bs)):
                    self.rows[s][e] = self.free.pop(0)
                    self.head = (self.head + 1) % self.NB
                for p in range(c, c + n):
                    slots.append(self.rows[s][p // bs] * bs + p % bs)
                    pos.append(p)
                    seqs.append(s)
                self.lens[s] += n
            start.append(len(slots))
        fill = T - len(slots)
        return start, slots + [-1] * fill, pos + [0] * fill, seqs + [-1] * fill

    def release(self, finished=None, window=0, sinks=0):
        bs = self.bs
        for s in range(self.B):
            c = self.lens[s]
            if finished is not None and finished[s]:
                entries = range(-(-c // bs))
                self.lens[s] = 0
            else:
                entries = [e for e in range(-(-c // bs)) if window and e * bs >= sinks and (e + 1) * bs <= c - window + 1]
            for e in entries:
                if self.rows[s][e] >= 0:
                    self.free.append(self.rows[s][e])
                    self.rows[s][e] = -1

    def check(self, tables, lens, queue, state):
        assert tables.cpu().tolist() == self.rows
        assert lens.cpu().tolist() == self.lens
        head, n = state.cpu().tolist()
        assert (head, n) == (self.head, len(self.free))
        q = queue.cpu().numpy()
        assert q[(head + np.arange(n)) % self.NB].tolist() == self.free


def check_lists(o, start, slots, pos, seqs):
    assert o.query_start.cpu().tolist() == start
    assert o.slot_mapping.cpu().tolist() == slots
    assert o.positions.cpu().tolist() == pos
    assert o.seq_ids.cpu().tolist() == seqs


@pytest.mark.parametrize("B,mb,NB,bs,seed", [(1, 4, 4, 16, 0), (3, 10, 40, 1, 1), (7, 20, 100, 7, 2), (64, 30, 900, 16, 3),
                                             (300, 40, 5000, 32, 4), (1100, 12, 4000, 8, 5)])
def test_steps_in_place(B, mb, NB, bs, seed):
    rng = np.random.default_rng(seed)
    h = Host(B, mb, NB, bs, free=rng.permutation(NB).tolist(), head=int(rng.integers(0, NB)))
    tables, lens, queue, state = h.device()
    T = 2 * B + 3 * bs
    out = pkv.make_step_tables(B, T)._replace(context_lens=lens, queue_state=state)
    for step in range(12):
        new = np.where(rng.random(B) < 0.1, rng.integers(0, 3 * bs, B), rng.integers(0, 2, B))
        want = h.extend(new.tolist(), T)
        got = pkv.extend_tables(tables, lens, dev(new), queue, state, bs, T, out=out)
        check_lists(got, *want)
        h.check(tables, lens, queue, state)
        done = (rng.random(B) < 0.2).astype(np.int32)
        window, sinks = [(0, 0), (bs, 0), (2 * bs + 3, bs + 1), (1, 0)][step % 4]
        h.release(done.tolist(), window, sinks)
        pkv.release_tables(tables, lens, queue, state, bs, finished=dev(done), window=window, sinks=sinks)
        h.check(tables, lens, queue, state)
        if step % 5 == 4:
            h.release(None, 3, 1)
            pkv.release_tables(tables, lens, queue, state, bs, window=3, sinks=1)
            h.check(tables, lens, queue, state)
    assert pkv.device_status() in ((0, 0), (7, pkv.FLAG_BAD_CONTEXT))  # (rows that are full refuse more)


@pytest.mark.parametrize("T", [0, 1, 5, 2047, 2048, 2049, 4097, 30000])
def test_lists_of_every_length(T):
    # one CTA, two, and the largest cluster; tokens for all of the lists, for none, and for a part
    for new in ([T], [0, T // 3, 0, T - T // 3, 0], [max(0, T - 7)], [0, 0]):
        h = Host(len(new), 4000, 8100, 8, head=8000)
        tables, lens, queue, state = h.device()
        want = h.extend(new, T)
        o = pkv.extend_tables(tables, lens, dev(new), queue, state, 8, T)
        check_lists(o, *want)
        h.check(tables, o.context_lens, queue, o.queue_state)
        assert lens.cpu().tolist() == [0] * len(new) and state.cpu().tolist() == [8000, 8100]  # inputs as they were
    assert pkv.device_status() == (0, 0)


@pytest.mark.parametrize("free", [0, 1, 4, 5, 6, 9, 10])
@pytest.mark.parametrize("T", [40, 30, 12])
def test_who_is_refused(free, T):
    h = Host(6, 8, 40, 4, free=range(40))
    for s, c in enumerate([3, 4, 5, 0, 7, 2]):
        h.extend([c if i == s else 0 for i in range(6)], 100)
    h.free = h.free[:free]
    tables, lens, queue, state = h.device()
    new = [1, 1, 2, 9, 1, 15]  # needs no block, one, none, three, none, four
    want = h.extend(new, T)
    o = pkv.extend_tables(tables, lens, dev(new), queue, state, 4, T)
    check_lists(o, *want)
    h.check(tables, o.context_lens, queue, o.queue_state)
    assert pkv.device_status() == (0, 0)


def test_as_the_host_allocator():
    a = pkv.BlockAllocator(50, 4)
    queue, state = pkv.make_free_queue(50, reserve_null_block=True)
    tables = torch.full((5, 12), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(5, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(2)
    for step in range(8):
        new = rng.integers(0, 6, 5)
        assert all(a.extend(s, int(n)) for s, n in enumerate(new))
        o = pkv.extend_tables(tables, lens, dev(new), queue, state, 4, 40)
        lens, state = o.context_lens, o.queue_state
        for s in range(5):
            ids, n = a.table(s)
            assert lens[s].item() == n and tables[s, :len(ids)].cpu().tolist() == ids
        t = 0
        for s, n in enumerate(new):
            for i in range(n):
                assert o.slot_mapping[t].item() == a.slot(s, lens[s].item() - n + i)
                t += 1
        if step == 3:
            for s in (1, 4):
                a.release(s)
            pkv.release_tables(tables, lens, queue, state, 4, finished=dev([0, 1, 0, 0, 1]))
        head, n = state.cpu().tolist()
        assert queue.cpu().numpy()[(head + np.arange(n)) % 50].tolist() == a.free_queue()


def test_bad_lengths_and_rows():
    h = Host(5, 3, 20, 4)
    h.extend([4, 0, 12, 3, 0], 100)
    tables, lens, queue, state = h.device()
    bad = lens.clone()
    bad[1] = -3
    new = [1, 2, 1, -5, 4]  # a negative length, a full row, a negative number of tokens
    want = h.extend([1, 0, 0, 0, 4], 10)
    o = pkv.extend_tables(tables, bad, dev(new), queue, state, 4, 10)
    check_lists(o, *want)
    assert o.context_lens.cpu().tolist() == [5, -3, 12, 3, 4]
    assert pkv.device_status() == (7, pkv.FLAG_BAD_CONTEXT)
    huge = dev([2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 1])
    o = pkv.extend_tables(tables, o.context_lens, huge, queue, o.queue_state, 4, 10)
    assert o.query_start.cpu().tolist() == [0, 0, 0, 0, 0, 1]
    assert pkv.device_status() == (7, pkv.FLAG_BAD_CONTEXT)


def test_bad_entries_and_queues():
    h = Host(2, 4, 10, 4)
    h.extend([2, 4], 100)
    tables, lens, queue, state = h.device()
    broken = tables.clone()
    broken[0, 0] = 10
    o = pkv.extend_tables(broken, lens, dev([1, 1]), queue, state, 4, 4)
    assert o.slot_mapping.cpu().tolist() == [-1, 2 * 4, -1, -1] and o.seq_ids.cpu().tolist() == [0, 1, -1, -1]
    assert pkv.device_status() == (7, pkv.FLAG_BAD_BLOCK_ID)
    odd = queue.clone()
    odd[2] = 77
    o = pkv.extend_tables(tables.clone(), lens, dev([1, 1]), odd, state, 4, 2)
    assert o.slot_mapping.cpu().tolist() == [tables[0, 0].item() * 4 + 2, -1]
    assert pkv.device_status() == (7, pkv.FLAG_BAD_QUEUE)
    for wrong in ([-1, 3], [10, 3], [0, 11], [0, -1]):
        kept = tables.clone()
        o = pkv.extend_tables(kept, lens, dev([1, 1]), queue, dev(wrong), 4, 2)
        assert o.query_start.cpu().tolist() == [0, 1, 1] and torch.equal(kept, tables)
        assert pkv.device_status() == (7, pkv.FLAG_BAD_QUEUE)
        was = dev(wrong)
        pkv.release_tables(kept, lens, queue, was, 4, finished=dev([1, 1]))
        assert torch.equal(kept, tables) and was.cpu().tolist() == wrong
        assert pkv.device_status() == (7, pkv.FLAG_BAD_QUEUE)
    full = dev([3, 9])  # nine of ten free, and two come back
    pkv.release_tables(tables, lens, queue, full, 4, finished=dev([1, 1]))
    assert full.cpu().tolist() == [3, 9] and lens.cpu().tolist() == [2, 4]
    assert pkv.device_status() == (7, pkv.FLAG_BAD_QUEUE)


def test_largest_batch_and_long_rows():
    B, bs = 8192, 16
    h = Host(B, 3, 3 * B, bs)
    tables, lens, queue, state = h.device()
    new = [(i * 7) % 40 for i in range(B)]
    T = sum(new) + 11
    want = h.extend(new, T)
    o = pkv.extend_tables(tables, lens, dev(new), queue, state, bs, T)
    check_lists(o, *want)
    done = [i % 3 == 0 for i in range(B)]
    h.release(done, 5, 16)
    lens = o.context_lens
    pkv.release_tables(tables, lens, queue, o.queue_state, bs, finished=dev(done), window=5, sinks=16)
    h.check(tables, lens, queue, o.queue_state)
    h = Host(2, 40000, 70000, 2, head=12345)
    tables, lens, queue, state = h.device()
    want = h.extend([60001, 77777], 150000)
    o = pkv.extend_tables(tables, lens, dev([60001, 77777]), queue, state, 2, 150000)
    check_lists(o, *want)
    h.release(None, 100, 50)
    lens = o.context_lens
    pkv.release_tables(tables, lens, queue, o.queue_state, 2, window=100, sinks=50)
    h.check(tables, lens, queue, o.queue_state)
    assert pkv.device_status() == (0, 0)


def test_no_sequences():
    tables = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    queue, state = pkv.make_free_queue(9)
    o = pkv.extend_tables(tables, none, none, queue, state, 4, 3)
    assert o.query_start.cpu().tolist() == [0] and o.slot_mapping.cpu().tolist() == [-1] * 3 and o.queue_state.cpu().tolist() == [0, 9]
    pkv.release_tables(tables, none, queue, state, 4, window=3)
    assert pkv.device_status() == (0, 0)


def test_refuses():
    h = Host(3, 4, 20, 4)
    tables, lens, queue, state = h.device()
    new = dev([1, 1, 1])
    good = (tables, lens, new, queue, state, 4, 5)
    for i in range(5):
        bad = list(good)
        bad[i] = bad[i].cpu()
        with pytest.raises(ValueError):
            pkv.extend_tables(*bad)
        bad[i] = good[i].long()
        with pytest.raises(ValueError):
            pkv.extend_tables(*bad)
    out = pkv.make_step_tables(3, 5)
    for bad in (pkv.make_step_tables(2, 5), pkv.make_step_tables(3, 6), out._replace(positions=out.slot_mapping),
                out._replace(context_lens=new), out._replace(queue_state=lens[:2]), out._replace(query_start=queue[:4])):
        with pytest.raises((ValueError, pkv.KVError)):
            pkv.extend_tables(*good, out=bad)
    with pytest.raises(pkv.KVError):
        pkv.extend_tables(*good[:5], 0, 5)
    for kw in (dict(window=-1), dict(sinks=-1), dict(finished=new.long()), dict(finished=new[:2])):
        with pytest.raises(ValueError):
            pkv.release_tables(tables, lens, queue, state, 4, **kw)
    with pytest.raises(pkv.KVError):
        pkv.release_tables(tables, lens, queue, state, 4, finished=lens)
