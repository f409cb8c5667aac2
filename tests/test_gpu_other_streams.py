"""GPU tests of calls that are given a stream other than torch's current one, and make a tensor of their own.

The current stream is kept busy for some milliseconds, so that whatever a call leaves on it comes late."""
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv
from test_gpu_append_rope import Case
from test_gpu_shared_prefix import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.empty_cache()


class Busy:
    """Matrix products on the stream that is current at the call."""

    def __init__(self):
        self.a = torch.randn((4096, 4096), device="cuda").half()
        self.c = torch.empty_like(self.a)
        torch.mm(self.a, self.a, out=self.c)
        torch.cuda.synchronize()

    def __call__(self):
        for _ in range(60):
            torch.mm(self.a, self.a, out=self.c)


@pytest.fixture(scope="module")
def busy():
    return Busy()


def _handles(side):
    return [side, side.cuda_stream, torch.cuda.ExternalStream(side.cuda_stream)]


@pytest.mark.parametrize("which", range(3))
def test_new_query_rows_with_padding(busy, which):
    c = Case(300, 8, 2, 128, 128, "bf16", packed=True)
    ids = torch.arange(300, dtype=torch.int32, device="cuda")
    ids[[7, 299]] = -1
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    q_out = c.run(seq_ids=ids, stream=_handles(side)[which])
    side.synchronize()
    torch.cuda.synchronize()
    c.check(q_out, ids)
    assert bool((q_out[[7, 299]] == 0).all())


def test_new_query_rows_without_padding(busy):
    c = Case(64, 8, 2, 128, 64, "f16")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    q_out = c.run(stream=side)
    torch.cuda.synchronize()
    c.check(q_out)


@pytest.mark.parametrize("axes", [1, 3])
def test_positions_that_are_copied(busy, axes):
    """Columns of [tokens, axes], copied into rows: the copy comes before the kernel, and its memory stays until then."""
    c = Case(500, 8, 2, 64, 64, "bf16", axes=axes)
    base = torch.full((500, axes + 2), 9, dtype=torch.int32, device="cuda")
    base[:, 1:axes + 1] = c.pos.t()
    keep = c.pos
    c.pos = base[:, 1:axes + 1].t()
    q_out = torch.empty_like(c.q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    with torch.cuda.stream(side):
        busy()
    c.run(q_out=q_out, stream=side)
    late = [torch.full((axes, 500), 77, dtype=torch.int32, device="cuda") for _ in range(8)]  # may take freed memory
    torch.cuda.synchronize()
    c.pos = keep
    c.check(q_out)
    assert all(bool((x == 77).all()) for x in late)


def test_the_default_stream_by_number(busy):
    c = Case(300, 4, 2, 128, 128, "f16")
    ids = torch.arange(300, dtype=torch.int32, device="cuda")
    ids[3] = -1
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        busy()
        q_out = c.run(seq_ids=ids, stream=0)
    torch.cuda.synchronize()
    c.check(q_out, ids)
    assert bool((q_out[3] == 0).all())


def test_a_forked_stream_in_a_captured_graph():
    c = Case(40, 8, 2, 128, 128, "bf16", axes=2)
    ids = torch.arange(40, dtype=torch.int32, device="cuda")
    ids[5] = -1
    base = c.pos.t().contiguous()
    keep, c.pos = c.pos, base.t()
    c.run(seq_ids=ids)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        q_out = c.run(seq_ids=ids, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    c.q.normal_()
    c.k.normal_()
    base.add_(31)
    c.pool.buffer.fill_(0x2B)
    graph.replay()
    torch.cuda.synchronize()
    c.pos = keep + 31
    c.check(q_out, ids)
    assert bool((q_out[5] == 0).all())


def test_outputs_filled_before_the_other_stream_waits():
    """The order that a caller has to keep: fill, let the other stream wait, call, wait for it."""
    c = Case(19, 8, 2, 128, 128, "bf16")
    side = torch.cuda.Stream()
    q_out = torch.full_like(c.q, float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    c.run(q_out=q_out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    c.check(q_out)
    assert pkv.device_status() == (0, 0)


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_prefix_attention_with_tensors_of_its_own(busy, fp8):
    """out and workspace are made by the call: what the current stream still does with their memory, or does with memory
    that it takes after the call, does not reach them."""
    b = Batch([9, 4], [700, 2000], [700 + 30 * i for i in range(9)] + [2000, 2100, 2500, 1999], "bf16", 4, 4, 128, fp8=fp8)
    n = b.workspace().numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # Memory that is free for the current stream's next tensors, and that the stream has yet to write.
    busy()
    early = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
    early += [torch.full(b.q.shape, float("nan"), dtype=torch.float32, device="cuda") for _ in range(3)]
    del early
    with torch.cuda.stream(side):
        busy()
    out = pkv.paged_shared_prefix_attention(b.q, b.kc, b.vc, b.tables, b.ctx, b.starts, b.plens, b.scale,
                                            out_dtype=torch.float32, stream=side, **b.scales)
    late = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    b.check(out)
    assert all(bool((x == 0x55).all()) for x in late)


def test_shared_prefix_attention_on_a_forked_stream_in_a_captured_graph():
    b = Batch([6, 3], [800, 320], [800 + 50 * i for i in range(6)] + [320, 400, 330], "f16", 4, 2, 128)
    b.run()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        out = pkv.paged_shared_prefix_attention(b.q, b.kc, b.vc, b.tables, b.ctx, b.starts, b.plens, b.scale,
                                                out_dtype=torch.float32, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    b.q.normal_()
    graph.replay()
    torch.cuda.synchronize()
    b.check(out)


def test_shared_prefix_out_filled_before_the_other_stream_waits():
    b = Batch([6], [800], [800 + 50 * i for i in range(6)], "bf16", 4, 2, 128)
    ws, side = b.workspace(), torch.cuda.Stream()
    out = torch.full(b.q.shape, float("nan"), dtype=torch.float32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    b.run(workspace=ws, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b.check(out)


class Cache:
    """One layer's cache with sequences of these lengths in blocks of any order."""

    def __init__(self, ctx, Hq=8, Hkv=2, D=128, bs=16, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.D, self.bs, self.dt = Hq, Hkv, D, bs, dtype
        n = [-(-c // bs) for c in ctx]
        self.NB = sum(n) + 3
        perm = torch.randperm(self.NB, generator=g, device="cuda", dtype=torch.int32).cpu()
        self.tables = torch.full((len(ctx), max(n)), -1, dtype=torch.int32)
        at = 0
        for s, m in enumerate(n):
            self.tables[s, :m] = perm[at:at + m]
            at += m
        self.tables = self.tables.cuda()
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.kc, self.vc = (torch.randn((self.NB, Hkv, bs, D), generator=g, device="cuda").to(dtype) for _ in range(2))
        self.new = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(dtype)  # noqa: E731


def _early_and_busy(busy, sizes, side):
    """Freed memory that the current stream has yet to write, and both streams busy."""
    torch.cuda.synchronize()
    busy()
    early = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    del early
    with torch.cuda.stream(side):
        busy()


@pytest.mark.parametrize("append", [False, True])
def test_decode_attention_with_tensors_of_its_own(busy, append):
    """The counters of the merge are zeroed before the kernel counts on them."""
    c = Cache([4000, 900, 17, 2500])
    q, k, v = c.new(4, c.Hq, c.D), c.new(4, c.Hkv, c.D), c.new(4, c.Hkv, c.D)
    scale = c.D ** -0.5

    def call(**kw):
        if append:
            return pkv.paged_decode_append_attention(q, k, v, c.kc, c.vc, c.tables, c.ctx, scale, **kw)
        return pkv.paged_decode_attention(q, c.kc, c.vc, c.tables, c.ctx, scale, **kw)

    want = call()
    n = pkv.workspace_bytes(4, c.Hq, c.Hkv, c.D)
    side = torch.cuda.Stream()
    _early_and_busy(busy, (n, q.nbytes), side)
    got = call(stream=side)
    late = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert pkv.device_status() == (0, 0)
    assert torch.equal(got, want)
    assert all(bool((x == 0x55).all()) for x in late)


def test_prefill_attention_and_slots_with_tensors_of_their_own(busy):
    c = Cache([300, 129, 700])
    starts = torch.tensor([0, 100, 129, 329], dtype=torch.int32, device="cuda")
    q = c.new(329, c.Hq, c.D)

    def call(**kw):
        return (pkv.slot_mapping(c.tables, c.ctx, c.bs, c.NB, **kw),
                pkv.slot_mapping_varlen(c.tables, starts, c.ctx, c.bs, c.NB, num_tokens=329, **kw),
                pkv.paged_prefill_attention(q, c.kc, c.vc, c.tables, starts, c.ctx, c.D ** -0.5, **kw))

    want = call()
    side = torch.cuda.Stream()
    _early_and_busy(busy, (16, 329 * 4, 65536, q.nbytes), side)
    got = call(stream=side)
    late = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in (512, 2048, 65536) for _ in range(4)]
    torch.cuda.synchronize()
    assert pkv.device_status() == (0, 0)
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert all(bool((x == 0x55).all()) for x in late)


def test_swap_of_listed_blocks_that_are_copied(busy):
    pool = pkv.KVPool(2, 12, 16, 2, 64, torch.float16)
    pool.buffer.copy_(torch.randint(0, 256, pool.buffer.shape, dtype=torch.uint8, device="cuda"))
    ids = torch.tensor([[3, 0], [11, 1], [5, 2]], dtype=torch.int32, device="cuda")[:, 0]
    want = pool.swap_out(ids)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    got = pool.swap_out(ids, stream=side)
    side.synchronize()
    n = pool.swap_bytes(3)
    assert torch.equal(got[:n], want[:n])
    torch.cuda.synchronize()
