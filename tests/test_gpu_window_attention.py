"""GPU tests of the windowed attention, of single tokens and of chunks, against the formula in 64 bits.

Tolerance of an fp32 output.  A score sums D exact products in fp32: off by at
most E = D * 2^-24 * sum_d |q_d k_d| * |scale| (and twice that with its scaling).
A weight is then off by 2 E relatively, by 2^-22 from the exponential and by
2^-16 from its two half-precision parts; numerator and denominator sum n terms
in fp32, n * 2^-24 each.  With A = sum p |v| the output is within
A * (4 E + 2^-15 + 2 n 2^-24).  In a chunk with a 16-bit output a weight may be
held in one part, off by half a step of q's type: A * eps / 2 more.  A 16-bit
output adds half a step of its own.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
KS, VS = 1 / 56, 1 / 44


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.empty_cache()


class Batch:
    """ctx: cached tokens of each sequence, the new ones included; new: new tokens of each (None: one query token of
    each, for the decode call; a sequence of length 0 then has a query row too).  Table entries that no query sees are
    -1, and every cached value that none sees is NaN."""

    def __init__(self, ctx, window, sinks=0, new=None, dtype="bf16", G=4, Hkv=2, D=128, bs=16, fp8=False, seed=0, spread=1.0,
                 pad=0, entries=-1):
        g = torch.Generator(device="cuda").manual_seed(seed + 17)
        rng = np.random.default_rng(seed)
        B = len(ctx)
        self.decode, self.new = new is None, [1 if c else 0 for c in ctx] if new is None else new
        self.ctx_list, self.window, self.sinks = list(ctx), window, sinks
        self.B, self.G, self.Hkv, self.D, self.bs, self.fp8 = B, G, Hkv, D, bs, fp8
        mb = max(1, max(-(-c // bs) for c in ctx))
        seen = np.zeros((B, mb * bs), bool)
        for s, (c, n) in enumerate(zip(ctx, self.new)):
            if n:
                seen[s, max(0, c - n + 1 - window):c] = True
                seen[s, :min(sinks, c)] = True
        blocks = seen.reshape(B, mb, bs).any(-1)
        NB = int(blocks.sum()) + 5
        perm = rng.permutation(NB).astype(np.int32)
        t = np.full((B, mb), entries, np.int32)
        t[blocks] = perm[:int(blocks.sum())]
        used = np.zeros((NB, bs), bool)
        used[t[blocks]] = seen.reshape(B, mb, bs)[blocks]
        used = torch.from_numpy(used).cuda()[:, None, :, None]
        dt = DT[dtype]

        def cache(sd):
            x = torch.randn((NB, Hkv, bs, D), generator=g, device="cuda")
            if fp8:
                return torch.where(used, (x * sd).to(E4M3).view(torch.uint8), torch.tensor(0x7F, dtype=torch.uint8, device="cuda")).view(E4M3)
            return torch.where(used, x.to(dt), torch.tensor(float("nan"), dtype=dt, device="cuda"))

        self.kc, self.vc = cache(56), cache(44)
        rows = B if self.decode else sum(self.new)
        self.q = (torch.randn((rows + pad, Hkv * G, D), generator=g, device="cuda") * spread).to(dt)
        self.start_list = [0, *np.cumsum(self.new).tolist()]
        self.tables = torch.from_numpy(t).cuda()
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.start = torch.tensor(self.start_list, dtype=torch.int32, device="cuda")
        self.scale = 1 / D ** 0.5
        self.scales = dict(k_scale=KS, v_scale=VS) if fp8 else {}

    def workspace(self, **opts):
        if self.decode:
            return pkv.make_workspace(self.B, self.G * self.Hkv, self.Hkv, self.D, **opts)
        n = pkv.window_prefill_workspace_bytes(self.B, self.q.shape[0], self.G * self.Hkv, self.Hkv, self.D)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, out_dtype=torch.float32, window=None, sinks=None, **kw):
        kw.setdefault("out", torch.full(self.q.shape, 7.0, dtype=out_dtype, device="cuda"))
        opts = {k: kw[k] for k in ("separate_reduce", "num_ctas", "ctas_per_sm", "consumer_warps", "kernel", "heads_per_stage") if k in kw}
        kw.setdefault("workspace", self.workspace(**opts))
        window, sinks = self.window if window is None else window, self.sinks if sinks is None else sinks
        if self.decode:
            return pkv.paged_window_decode_attention(self.q, self.kc, self.vc, self.tables, self.ctx, self.scale, window, sinks,
                                                     out_dtype=out_dtype, **self.scales, **kw)
        return pkv.paged_window_prefill_attention(self.q, self.kc, self.vc, self.tables, self.start, self.ctx, self.scale, window,
                                                  sinks, out_dtype=out_dtype, **self.scales, **kw)

    def rows(self, s, cache, scale):
        """All cached rows of sequence s in float64, [Hkv, ctx, D]; 0 where nothing is held."""
        c = self.ctx_list[s]
        blk = self.tables[s, :-(-c // self.bs)].long()
        x = cache[blk.clamp(0, cache.shape[0] - 1)]
        x = x.float().double() * scale if self.fp8 else x.double()
        x = torch.where((blk >= 0)[:, None, None, None] & (blk < cache.shape[0])[:, None, None, None], x, torch.zeros_like(x))
        return x.transpose(0, 1).flatten(1, 2)[:, :c]

    def expected(self):
        """(output, bound) in float64; rows of no sequence: 7, as run() leaves them (decode: 0)."""
        out = torch.full(self.q.shape, 0.0 if self.decode else 7.0, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        one_part = 0.0 if self.decode else torch.finfo(self.q.dtype).eps / 2
        for s, (c, n) in enumerate(zip(self.ctx_list, self.new)):
            if not n:
                continue
            at = slice(s, s + 1) if self.decode else slice(self.start_list[s], self.start_list[s] + n)
            p = torch.arange(c - n, c, device="cuda")[:, None]
            j = torch.arange(c, device="cuda")
            seen = (j <= p) & ((j > p - self.window) | (j < self.sinks))
            k, v = self.rows(s, self.kc, KS if self.fp8 else 1), self.rows(s, self.vc, VS if self.fp8 else 1)
            any_row = seen.any(0)[None, :, None]
            k, v = torch.where(any_row, k, torch.zeros_like(k)), torch.where(any_row, v, torch.zeros_like(v))
            q = self.q[at].double().view(n, self.Hkv, self.G, self.D).permute(1, 2, 0, 3)  # [Hkv, G, n, D]
            x = (q @ k[:, None].mT * self.scale).masked_fill(~seen, -torch.inf)
            w = torch.softmax(x, -1)
            out[at] = (w @ v[:, None]).permute(2, 0, 1, 3).reshape(n, -1, self.D)
            err = (self.D * 2.0 ** -24 * abs(self.scale) * (q.abs() @ k[:, None].abs().mT).masked_fill(~seen, 0).amax(-1, keepdim=True))
            a = w @ v[:, None].abs()
            bound = a * (4 * err + 2.0 ** -15 + 2 * c * 2.0 ** -24)
            tol[at] = bound.permute(2, 0, 1, 3).reshape(n, -1, self.D)
            if one_part:
                self.part = getattr(self, "part", torch.zeros_like(out))
                self.part[at] = (a * one_part).permute(2, 0, 1, 3).reshape(n, -1, self.D)
        return out, tol

    def check(self, out, what=""):
        assert pkv.device_status() == (0, 0), what
        ref, tol = self.expected()
        if out.dtype != torch.float32:
            info = torch.finfo(out.dtype)
            tol = tol + (0 if self.decode else self.part)
            tol = tol + torch.where(tol > 0, info.eps / 2 * (ref.abs() + tol) + info.smallest_normal * info.eps / 2, torch.zeros_like(tol))
        assert torch.isfinite(out).all(), what
        off = (out.double() - ref).abs() - tol
        assert float(off.max()) <= 0, f"{what}: {float(off.max()):.3e} past the bound"


# Around a window of 40 and 20 first tokens in blocks of 16: nothing, one token, all in sight, the window leaving the
# first tokens by one, block borders on both sides of the gap, far away.
LENGTHS = [0, 1, 16, 39, 40, 41, 56, 59, 60, 61, 62, 72, 73, 80, 81, 200, 1000, 0]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_decode(dtype, D, G):
    b = Batch(LENGTHS, 40, 20, dtype=dtype, G=G, D=D, seed=G)
    b.check(b.run())


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [16, 32, 48, 64])
def test_decode_e4m3(G, dtype, bs):
    b = Batch(LENGTHS, 40, 20, dtype=dtype, G=G, bs=bs, fp8=True, seed=G)
    b.check(b.run())


@pytest.mark.parametrize("bs", [8, 16, 24, 32, 48, 64, 128, 192])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 16), (33, 0), (64, 4), (100, 33), (129, 200), (1 << 30, 0),
                                          (50, 1 << 30), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_decode_sizes(bs, window, sinks):
    b = Batch([0, 1, 5, 17, 63, 64, 65, 100, 193, 257, 511, 700], window, sinks, dtype="f16", bs=bs, seed=bs)
    b.check(b.run())


@pytest.mark.parametrize("opts", [dict(separate_reduce=True), dict(num_ctas=1), dict(num_ctas=7), dict(heads_per_stage=1),
                                  dict(consumer_warps=1), dict(kernel="ffma"), dict(ctas_per_sm=2), dict(early_reads=True)])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_options(opts, fp8):
    if fp8 and opts.get("kernel") == "ffma":
        pytest.skip("an E4M3 cache is read by the tensor-core kernel only")
    b = Batch([700, 3, 0, 512, 90, 2000], 300, 5, dtype="bf16", Hkv=4, fp8=fp8)
    b.check(b.run(**opts))


def test_decode_outputs_and_repetition():
    b = Batch([3000, 150, 1, 0, 4097, 2222, 64], 1024, 4, dtype="bf16", Hkv=8, G=4, bs=32)
    ws = b.workspace()
    first = b.run(torch.bfloat16, workspace=ws)
    b.check(first)
    for _ in range(3):
        assert torch.equal(first, b.run(torch.bfloat16, workspace=ws))
    fresh = pkv.paged_window_decode_attention(b.q, b.kc, b.vc, b.tables, b.ctx, b.scale, 1024, 4)
    assert torch.equal(first, fresh) and fresh.dtype == torch.bfloat16


def test_decode_whole_context_is_the_plain_decode():
    b = Batch([3000, 150, 1, 0, 999], 1 << 20, 0, dtype="f16", Hkv=4)
    full = pkv.paged_decode_attention(b.q, b.kc, b.vc, b.tables, b.ctx, b.scale)
    b.check(full)
    for sinks in (0, 4, 5000):
        # with a launch shape the same kernel, bit for bit; else one that sums in another order
        assert torch.equal(full, b.run(torch.float16, sinks=sinks, consumer_warps=8))
        b.check(b.run(torch.float16, sinks=sinks))


def test_decode_many_sequences():
    rng = np.random.default_rng(5)
    b = Batch(rng.integers(0, 3000, 300).tolist(), 129, 3, dtype="bf16", G=8, Hkv=1)
    b.check(b.run(torch.bfloat16))
    b.check(b.run(torch.bfloat16, consumer_warps=8))


@pytest.mark.parametrize("shape", [dict(consumer_warps=8), dict(num_ctas=40)])
@pytest.mark.parametrize("dtype,D,G,bs,fp8", [("f16", 64, 2, 16, False), ("bf16", 128, 8, 32, False), ("bf16", 128, 4, 16, True),
                                              ("f16", 128, 8, 48, True), ("bf16", 128, 8, 16, True)])
def test_decode_with_a_launch_shape(shape, dtype, D, G, bs, fp8):
    """The persistent kernel, at sizes that otherwise go to the one for small calls."""
    for window, sinks in ((40, 20), (1, 0), (300, 5)):
        b = Batch(LENGTHS + [3000], window, sinks, dtype=dtype, G=G, D=D, bs=bs, fp8=fp8)
        b.check(b.run(**shape))


@pytest.mark.parametrize("B", [1, 2, 5, 40])
@pytest.mark.parametrize("dtype,bs,fp8", [("bf16", 16, False), ("f16", 128, False), ("bf16", 64, True)])
def test_decode_small_calls(B, dtype, bs, fp8):
    """Clusters of every size: few and many heads, more blocks than warps."""
    for Hkv in (1, 8):
        b = Batch([(i * 977) % 5000 + 1 for i in range(B)], 2000, 17, dtype=dtype, Hkv=Hkv, bs=bs, fp8=fp8)
        b.check(b.run())


@pytest.mark.parametrize("scale", [0.0, -0.7, 3.0])
def test_scales_of_any_sign(scale):
    for new in (None, [1, 30, 64]):
        b = Batch([100, 33, 70], 25, 2, new=new)
        b.scale = scale
        b.check(b.run())


@pytest.mark.parametrize("entries", [-1, 1 << 30, -(1 << 31)])
def test_entries_out_of_sight_are_not_read(entries):
    for new in (None, [3, 100, 1]):
        b = Batch([600, 517, 300], 64, 20, new=new, entries=entries)
        b.check(b.run())


def test_bad_entries_are_flagged():
    for new in (None, [3, 100]):
        b = Batch([600, 517], 64, 20, new=new)
        b.tables[0, 599 // 16] = b.kc.shape[0]
        b.run()
        assert pkv.device_status() == (7, pkv.FLAG_BAD_BLOCK_ID)


# ------------------------------------------------------------------ chunks

# (cached with the new tokens, new tokens): decoding rows, whole prompts, chunks that start inside the first tokens, at
# a tile's border, far behind; an empty sequence; a sequence without new tokens.
CHUNKS = [(1, 1), (0, 0), (20, 20), (300, 300), (41, 1), (500, 1), (90, 33), (700, 128), (64, 16), (333, 17), (50, 0), (1029, 65)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_chunks(dtype, D, G):
    b = Batch([c for c, _ in CHUNKS], 40, 20, new=[n for _, n in CHUNKS], dtype=dtype, G=G, D=D, seed=G, pad=3)
    b.check(b.run())
    b.check(b.run(DT[dtype]))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [1, 7, 16])
def test_chunks_f32(D, bs):
    b = Batch([c for c, _ in CHUNKS], 40, 20, new=[n for _, n in CHUNKS], dtype="f32", D=D, bs=bs, pad=2)
    b.check(b.run())


@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [16, 32, 48, 128])
def test_chunks_e4m3(G, dtype, bs):
    b = Batch([c for c, _ in CHUNKS], 40, 20, new=[n for _, n in CHUNKS], dtype=dtype, G=G, bs=bs, fp8=True, pad=1)
    b.check(b.run())
    b.check(b.run(DT[dtype]))


@pytest.mark.parametrize("D,bs", [(128, 16), (128, 32), (128, 48), (128, 64), (128, 128), (128, 192), (64, 16), (64, 80)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (16, 16), (33, 0), (64, 4), (100, 33), (129, 200), (1 << 30, 0),
                                          (50, 1 << 30), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_chunk_sizes(D, bs, window, sinks):
    ctx, new = [257, 5, 700, 64, 511, 300], [257, 1, 40, 64, 100, 7]
    b = Batch(ctx, window, sinks, new=new, dtype="f16", D=D, bs=bs, seed=bs)
    b.check(b.run())
    b.check(b.run(torch.float16))


def test_chunk_whole_context_matches_the_plain_prefill():
    b = Batch([300, 77, 700], 1 << 20, 0, new=[300, 7, 100], dtype="bf16", Hkv=4)
    full = pkv.paged_prefill_attention(b.q, b.kc, b.vc, b.tables, b.start, b.ctx, b.scale, out_dtype=torch.float32)
    b.check(full)
    for sinks in (0, 4, 5000):
        b.check(b.run(sinks=sinks))


def test_long_chunk():
    b = Batch([5000, 2100], 1024, 4, new=[3000, 2100], dtype="bf16", G=4, Hkv=2, pad=5)
    b.check(b.run(torch.bfloat16))


def test_large_scores_and_late_maxima():
    # The largest score of a row in its last tile, and scores far apart: the sums are rescaled at every step.
    for dtype in ("f16", "bf16"):
        b = Batch([900, 400], 500, 4, new=[300, 400], dtype=dtype, spread=6.0)
        ramp = torch.linspace(0.05, 3.0, 16, device="cuda")[None, None, :, None]
        b.kc = (b.kc.float() * ramp).to(b.kc.dtype)
        b.check(b.run())
        b.check(b.run(DT[dtype]))


@pytest.mark.parametrize("D,dtype,fp8", [(128, "bf16", False), (128, "f16", False), (64, "bf16", False), (128, "f32", False)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_chunk_rows_are_apart(D, dtype, fp8, value):
    """A value that is no number in one token's K or V stays out of the rows that do not see it."""
    b = Batch([300], 40, 2, new=[120], dtype=dtype, D=D, fp8=fp8)
    clean, bound = b.expected()
    at = 230  # seen by the tokens at positions 230 .. 269: rows 50 .. 89
    blk, off = int(b.tables[0, at // b.bs]), at % b.bs
    for cache in (b.kc, b.vc):
        kept = cache[blk, 0, off, 5].clone()
        cache[blk, 0, off, 5] = value
        out = b.run().double()
        cache[blk, 0, off, 5] = kept
        assert pkv.device_status() == (0, 0)
        others = torch.tensor([r for r in range(120) if not 50 <= r < 90], device="cuda")
        assert torch.isfinite(out[others]).all()
        assert float(((out - clean).abs() - bound)[others].max()) <= 0
        assert float(((out - clean).abs() - bound)[:, b.G:].max()) <= 0  # the other KV head
        if cache is b.vc or value != value:  # (an infinite K element may leave a weight of 0 or 1)
            assert not torch.isfinite(out[50:90, :b.G, 5]).any()


def test_bad_lengths_are_flagged_and_skipped():
    b = Batch([100, 50, 60], 30, 2, new=[20, 10, 5])
    b.ctx[1] = 5  # fewer than its new tokens
    out = b.run()
    assert pkv.device_status() == (7, pkv.FLAG_BAD_CONTEXT)
    ref, tol = b.expected()
    keep = [*range(20), *range(30, 35)]
    assert float(((out.double() - ref).abs() - tol)[keep].max()) <= 0
    assert bool((out[20:30] == 7).all())


def test_other_stream_graph_and_threads():
    for new in (None, [30, 1, 200]):
        b = Batch([400, 33, 200], 64, 4, new=new, dtype="bf16")
        ws = b.workspace()
        out = torch.empty(b.q.shape, dtype=torch.bfloat16, device="cuda")
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        b.run(torch.bfloat16, workspace=ws, out=out, stream=side)
        side.synchronize()
        want = out.clone()
        b.check(out) if b.decode else None
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run(torch.bfloat16, workspace=ws, out=out)
        for _ in range(2):
            b.q.copy_(b.q.flip(0)) if b.decode else None
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            if not b.decode:
                assert torch.equal(out, want)
        if b.decode:
            assert torch.equal(out, want)


def test_refuses_host_and_wrong_tensors():
    b = Batch([100, 50], 30, 2, new=[20, 10])
    d = Batch([100, 50], 30, 2)
    for make, call in ((b, pkv.paged_window_prefill_attention), (d, pkv.paged_window_decode_attention)):
        lists = (make.start, make.ctx) if make is b else (make.ctx,)
        good = [make.q, make.kc, make.vc, make.tables, *lists]
        for i in range(len(good)):
            bad = list(good)
            bad[i] = bad[i].cpu()
            with pytest.raises(ValueError):
                call(*bad, make.scale, 30, 2)
        for kw in (dict(window=0), dict(window=-3), dict(sinks=-1), dict(out_dtype=torch.float16),
                   dict(out=torch.empty(3, device="cuda")), dict(workspace=make.workspace()[::2])):
            args = dict(window=30, sinks=2)
            args.update(kw)
            with pytest.raises((ValueError, pkv.KVError)):
                call(*good, make.scale, **args)
        with pytest.raises(ValueError):
            call(make.q.half(), *good[1:], make.scale, 30)
        with pytest.raises(ValueError):
            call(make.q[:, :, :64], *good[1:], make.scale, 30)


@pytest.mark.parametrize("D,dtype,fp8", [(128, "bf16", False), (64, "f16", False), (128, "f16", True)])
def test_chunk_of_nan_values(D, dtype, fp8):
    """Every V that a chunk sees NaN: every row is NaN, and the call ends soon."""
    b = Batch([3000, 400], 700, 4, new=[2500, 400], dtype=dtype, D=D, Hkv=4, fp8=fp8)
    if fp8:
        b.q.fill_(float("nan"))
    else:
        b.vc.fill_(float("nan"))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    b.run(DT[dtype])
    start.record()
    out = b.run(DT[dtype])
    end.record()
    torch.cuda.synchronize()
    assert bool(out.isnan().all()) and pkv.device_status() == (0, 0)
    assert start.elapsed_time(end) < 1000.0


def test_chunk_with_one_nan_far_back():
    """Rows of 4,000 keys computed again, each 32 keys at a time, against the formula without the NaN's dimension."""
    b = Batch([4500], 4096, 4, new=[300], dtype="bf16", spread=2.0)
    clean, bound = b.expected()
    at = 4350  # seen by the rows from 150 on
    b.vc[int(b.tables[0, at // b.bs]), 1, at % b.bs, 7] = float("nan")
    out = b.run().double()
    off = (out - clean).abs() - bound
    off[150:, b.G:, 7] = -1
    assert float(off.max()) <= 0
    assert bool(out[150:, b.G:, 7].isnan().all())
