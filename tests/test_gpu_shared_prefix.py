"""GPU tests of the shared-prefix attention against the formula in 64 bits, sequence by sequence.

Tolerance of an fp32 output.  A score sums D exact products in fp32: off by at
most E = D * 2^-24 * sum_d |q_d k_d| * |scale| (and twice that with its scaling).
A weight is then off by 2 E relatively, by 2^-22 from the exponential and by
2^-16 from its two half-precision parts; numerator and denominator sum n terms
in fp32, n * 2^-24 each.  With A = sum p |v| the output is within
A * (4 E + 2^-15 + 2 n 2^-24).  A 16-bit output adds half a step.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
KS, VS = 1 / 56, 1 / 44


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.empty_cache()


class Batch:
    """sizes: sequences of each group; plens: prefix lengths; ctx: lengths (per sequence).
    before / after: sequences in no group.  Every cached value that no sequence reads is NaN."""

    def __init__(self, sizes, plens, ctx, dtype="bf16", G=4, Hkv=2, D=128, bs=16, fp8=False, seed=0, before=0, after=0,
                 spread=1.0, empty_groups=False):
        g = torch.Generator(device="cuda").manual_seed(seed + 17)
        rng = np.random.default_rng(seed)
        B = before + sum(sizes) + after
        assert len(ctx) == B
        self.B, self.G, self.Hkv, self.D, self.bs, self.fp8 = B, G, Hkv, D, bs, fp8
        starts = np.concatenate([[0], np.cumsum(sizes)]) + before
        group = [None] * B
        for i in range(len(sizes)):
            for s in range(starts[i], starts[i + 1]):
                group[s] = i
        shared = [p // bs for p in plens]
        members = [group[s] is not None and ctx[s] >= shared[group[s]] * bs for s in range(B)]
        mb = max(1, max(-(-c // bs) for c in ctx))
        need = sum(shared) + sum(-(-c // bs) for c in ctx)
        NB = need + 5
        perm = iter(rng.permutation(NB).astype(np.int32))
        shared_ids = [[next(perm) for _ in range(n)] for n in shared]
        t = np.full((B, mb), -1, np.int32)
        used = np.zeros((NB, bs), bool)
        for s, c in enumerate(ctx):
            n = -(-c // bs)
            pre = shared_ids[group[s]] if members[s] else []
            t[s, :n] = (pre + [next(perm) for _ in range(n - len(pre))])[:n]
            pos = np.arange(c)
            used[t[s, pos // bs], pos % bs] = True
        dt = DT[dtype]
        used = torch.from_numpy(used).cuda()[:, None, :, None]
        if fp8:
            self.kc, self.vc = ((torch.randn((NB, Hkv, bs, D), generator=g, device="cuda") * sd).to(E4M3) for sd in (56, 44))
        else:
            self.kc, self.vc = (torch.where(used, torch.randn((NB, Hkv, bs, D), generator=g, device="cuda").to(dt),
                                            torch.tensor(float("nan"), dtype=dt, device="cuda")) for _ in range(2))
        self.q = (torch.randn((B, Hkv * G, D), generator=g, device="cuda") * spread).to(dt)
        if empty_groups:  # the same groups with empty ones before, between and behind
            starts = np.repeat(starts, 2)
            plens = [x for p in plens for x in (999, p)] + [64]
        self.tables = torch.from_numpy(t).cuda()
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.starts = torch.from_numpy(starts.astype(np.int32)).cuda()
        self.plens = torch.tensor(plens, dtype=torch.int32, device="cuda")
        self.scale = 1 / D ** 0.5
        self.scales = dict(k_scale=KS, v_scale=VS) if fp8 else {}

    def workspace(self):
        n = pkv.shared_prefix_workspace_bytes(self.B, self.plens.shape[0], self.G * self.Hkv, self.Hkv, self.D)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, out_dtype=torch.float32, **kw):
        out = torch.full(self.q.shape, float("nan"), dtype=out_dtype, device="cuda")
        kw.setdefault("workspace", self.workspace())
        kw.setdefault("out", out)
        return pkv.paged_shared_prefix_attention(self.q, self.kc, self.vc, self.tables, self.ctx, self.starts, self.plens,
                                                 self.scale, out_dtype=out_dtype, **self.scales, **kw)

    def expected(self):
        """(output, bound) in float64."""
        out = torch.zeros(self.q.shape, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        for s, c in enumerate(self.ctx.tolist()):
            if c <= 0:
                continue
            blk = self.tables[s, :-(-c // self.bs)].long()

            def rows(cache, scale):
                x = cache.view(torch.uint8)[blk].view(E4M3).float().double() * scale if self.fp8 else cache[blk].double()
                return x.transpose(0, 1).flatten(1, 2)[:, :c]

            k, v = rows(self.kc, KS if self.fp8 else 1), rows(self.vc, VS if self.fp8 else 1)
            q = self.q[s].double().view(self.Hkv, self.G, self.D)
            p = torch.softmax(q @ k.mT * self.scale, -1)
            out[s] = (p @ v).flatten(0, 1)
            err = self.D * 2.0 ** -24 * (q.abs() @ k.abs().mT).amax(-1, keepdim=True) * abs(self.scale)
            tol[s] = ((p @ v.abs()) * (4 * err + 2.0 ** -15 + 2 * c * 2.0 ** -24)).flatten(0, 1)
        return out, tol

    def check(self, out, what=""):
        assert pkv.device_status() == (0, 0)
        ref, tol = self.expected()
        if out.dtype != torch.float32:
            info = torch.finfo(out.dtype)
            tol = tol + info.eps / 2 * (ref.abs() + tol) + info.smallest_normal * info.eps / 2
        off = (out.double() - ref).abs() - tol
        assert torch.isfinite(out).all(), what
        assert float(off.max()) <= 0, f"{what}: {float(off.max()):.3e} past the bound"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_groups(dtype, D, G):
    # prefixes: none, less than a block, one block, not a multiple, several tiles; tails of 0, 1, a block, more; lengths
    # inside the prefix, 0; a group of one; sequences in no group on both sides.
    sizes, plens = [3, 2, 1, 4, 5], [0, 15, 16, 203, 640]
    ctx = [33] + [5, 40, 70] + [1, 90] + [40] + [192, 193, 300, 0] + [640, 641, 656, 700, 639] + [17, 0]
    b = Batch(sizes, plens, ctx, dtype, G, 2, D, before=1, after=2, seed=G)
    b.check(b.run(), "fp32")
    b.check(b.run(DT[dtype]), dtype)


@pytest.mark.parametrize("bs", [16, 32, 48, 64, 112, 128, 256])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_block_sizes_and_heads(bs, Hkv):
    sizes, plens = [4, 3], [5 * bs + 3, 12 * bs]
    ctx = [5 * bs, 5 * bs + 1, 9 * bs - 1, 6 * bs] + [12 * bs + 5, 15 * bs, 12 * bs]
    b = Batch(sizes, plens, ctx, "f16", 4, Hkv, 64 if Hkv == 3 or bs > 200 else 128, bs=bs, seed=bs)
    b.check(b.run(), f"bs {bs}")


@pytest.mark.parametrize("G,members", [(8, 70), (4, 32), (4, 33), (1, 300), (8, 17), (2, 1)])
def test_row_tiles(G, members):
    """More than 128 query rows a KV head, and row tiles that end early."""
    ctx = [1000 + (37 * i) % 150 for i in range(members)]
    b = Batch([members], [960], ctx, "bf16", G, 2, 128, seed=members)
    b.check(b.run(torch.bfloat16), "rows")


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("plen", [16, 64, 80, 1024, 4097, 20000, 50000])
def test_prefix_lengths(dtype, D, plen):
    """From one run of 16 keys to a prefix split over many CTAs, each with many tiles."""
    ctx = [plen + x for x in (0, 1, 15, 16, 17, 100)]
    b = Batch([6], [plen], ctx, dtype, 4, 2, D, seed=plen)
    b.check(b.run(), f"prefix {plen}")


def test_long_chunks():
    """Many pairs and few CTAs for each: chunks of dozens of tiles."""
    b = Batch([5, 7], [16000, 9000], [16000 + 100 * i for i in range(5)] + [9000 + 11 * i for i in range(7)], "bf16", 2, 16, 128, bs=32)
    b.check(b.run(), "long chunks")


def test_many_groups():
    sizes = [2] * 40
    plens = [64 + 16 * (i % 7) for i in range(40)]
    ctx = [plens[i // 2] + 3 * i for i in range(80)]
    for empty in (False, True):
        b = Batch(sizes, plens, ctx, "f16", 4, 8, 128, empty_groups=empty)
        b.check(b.run(), f"empty groups {empty}")


def test_more_groups_than_plan_threads():
    """1100 groups (the plan takes them in turns), some of one short sequence."""
    n = 1100
    plens = [16 * (1 + i % 3) for i in range(n)]
    ctx = [plens[i] + i % 20 if i % 11 else i % 5 for i in range(n)]
    b = Batch([1] * n, plens, ctx, "bf16", 1, 1, 64)
    b.check(b.run(), "1100 groups")


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    """Sizes drawn over their ranges: many and few sequences, long and short prefixes and tails, any division of the SMs."""
    rng = np.random.default_rng(1000 + seed)
    n = int(rng.integers(1, 7))
    sizes = [int(x) for x in rng.integers(0, 40 if seed % 2 else 9, n)]
    bs = int(rng.choice([16, 32, 48, 64]))
    plens = [int(np.exp(rng.uniform(0, 9 if seed % 3 else 7))) for _ in range(n)]
    before, after = int(rng.integers(0, 3)), int(rng.integers(0, 3))
    top = int(np.exp(rng.uniform(0, 8)))
    ctx = [int(rng.integers(0, top + 1)) for _ in range(before)]
    for m, p in zip(sizes, plens):
        ctx += [p + int(rng.integers(0, top + 1)) if rng.random() < 0.9 else int(rng.integers(0, p + 1)) for _ in range(m)]
    ctx += [int(rng.integers(0, top + 1)) for _ in range(after)]
    fp8 = seed % 4 == 3
    b = Batch(sizes, plens, ctx, str(rng.choice(["f16", "bf16"])), int(rng.choice([1, 2, 4, 8])), int(rng.choice([1, 2, 3, 5, 8])),
              128 if fp8 else int(rng.choice([64, 128])), bs=bs, fp8=fp8, seed=seed, before=before, after=after) if ctx else None
    if b is not None:
        b.check(b.run(), f"seed {seed}")


def test_the_mixed_prefix_workload():
    """The workload of 64 sequences in groups of 8 with 2,048 shared tokens: as paged_decode_attention over the same tables."""
    from workloads import SPECS, make_placement, step_layer_values

    spec = SPECS["mixed_prefix_b64"]
    pl = make_placement(spec)
    pool = pkv.KVPool(1, pl.num_blocks, spec.block_size, spec.num_kv_heads, spec.head_dim, spec.torch_dtype)
    kc, vc = pool.layer(0)
    kc.normal_()
    vc.normal_()
    q = step_layer_values(spec, 64, 0, "cpu")[0].cuda()
    tables, ctx = torch.from_numpy(pl.block_tables).cuda(), torch.from_numpy(pl.context_lens).cuda()
    starts = torch.arange(0, 65, 8, dtype=torch.int32, device="cuda")
    plens = torch.full((8,), 2048, dtype=torch.int32, device="cuda")
    want = pkv.paged_decode_attention(q, kc, vc, tables, ctx, spec.attn_scale, out_dtype=torch.float32)
    got = pkv.paged_shared_prefix_attention(q, kc, vc, tables, ctx, starts, plens, spec.attn_scale, out_dtype=torch.float32)
    assert pkv.device_status() == (0, 0)
    # Both are within the tolerance above of the formula: A is below 1 and E below 2^-13 here, n up to 16,384.
    assert float((got - want).abs().max()) <= 2 * (4 * 2.0 ** -13 + 2.0 ** -15 + 2 * 16384 * 2.0 ** -24)


def test_two_streams_at_once():
    """Eager calls on two streams, each with a workspace of its own."""
    b = Batch([7, 5], [1000, 2500], [1000 + 40 * i for i in range(7)] + [2500 + 60 * i for i in range(5)], "f16", 4, 4, 128)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [b.workspace(), b.workspace()]
    outs = [torch.full(b.q.shape, float("nan"), dtype=torch.float32, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, w, o in zip(streams, spaces, outs):
            b.run(workspace=w, out=o, stream=st)
    torch.cuda.synchronize()
    for o in outs:
        b.check(o)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("G,bs", [(1, 16), (4, 32), (8, 48), (4, 128)])
def test_e4m3(dtype, G, bs):
    sizes, plens = [4, 9], [7 * bs, 2000]
    ctx = [7 * bs, 7 * bs + 1, 9 * bs, 3] + [2000 + 31 * i for i in range(9)]
    b = Batch(sizes, plens, ctx, dtype, G, 4, 128, bs=bs, fp8=True, seed=G)
    b.check(b.run(), "fp32")
    b.check(b.run(DT[dtype]), dtype)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.5])
def test_scales(scale):
    """Negative, zero, and scores so far apart that the running reference moves."""
    b = Batch([5], [1500], [1500, 1510, 1600, 1999, 2000], "bf16", 4, 2, 128)
    b.scale = scale
    b.check(b.run(), f"scale {scale}")


def test_growing_scores():
    """Scores that rise along the prefix move the reference in every tile."""
    b = Batch([4], [2048], [2100] * 4, "f16", 4, 1, 128)
    ramp = torch.linspace(0.02, 1, 2048, device="cuda")
    blk = b.tables[0, :128].long()
    unit = b.q[0, 0] / b.q[0, 0].float().norm()
    b.kc[blk] = (ramp.view(128, 1, 16, 1) * unit.float() * 12 + 0.1 * b.kc[blk].float()).half()
    b.scale = 0.7
    b.check(b.run(), "ramp")


def test_one_hot_and_minus_infinity():
    """Keys of -inf against a positive query weigh nothing, also where they fill a whole chunk or tile."""
    b = Batch([3], [1024], [1030] * 3, "bf16", 1, 1, 64)
    b.q[:] = b.q.abs() + 0.1
    blk = b.tables[0, :64].long()
    b.kc[blk[:40]] = float("-inf")
    out = b.run()
    assert pkv.device_status() == (0, 0)
    b.kc[blk[:40]] = -1e4  # finite and as good as -inf
    ref, tol = b.expected()
    assert float(((out.double() - ref).abs() - tol).max()) <= 0


def test_no_sharing_equals_plain_decode():
    """No groups, groups without a prefix, and every sequence too short: the tails do it all."""
    ctx = [100, 1, 0, 517, 64]
    b = Batch([2, 3], [0, 0], ctx, "bf16", 4, 2, 128)
    want = pkv.paged_decode_attention(b.q, b.kc, b.vc, b.tables, b.ctx, b.scale, out_dtype=torch.float32)
    got = [b.run()]
    b.plens[:] = 4096
    got.append(b.run())
    b.starts, b.plens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    got.append(b.run())
    for g in got:
        b.check(g)
        assert torch.allclose(g, want, atol=1e-5, rtol=1e-5)


def test_all_lengths_zero():
    b = Batch([3], [64], [0, 0, 0], "f16", 2, 2, 64)
    b.check(b.run())


@pytest.mark.parametrize("starts", [[0, 4, 3, 6], [0, 2, 7, 6], [-1, 2, 3, 6], [2, 1, 0, 0], [0, 2, 4, 100]])
def test_bad_groups_are_flagged_and_nothing_is_shared(starts):
    b = Batch([2, 2, 2], [64, 128, 32], [100, 101, 200, 201, 40, 50], "bf16", 4, 2, 128)
    b.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out = b.run()
    assert pkv.device_status() == (7, pkv.FLAG_BAD_GROUP)
    b.check(out)
    b.starts = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
    b.plens[1] = -5
    out = b.run()
    assert pkv.device_status() == (7, pkv.FLAG_BAD_GROUP)
    b.check(out)


def test_bad_blocks_and_lengths_are_flagged():
    b = Batch([3], [128], [140, 150, 160], "f16", 4, 2, 128)
    b.kc.nan_to_num_(0.0), b.vc.nan_to_num_(0.0)
    good = b.tables.clone()
    b.tables[:, 3] = 10 ** 6
    b.run()
    assert pkv.device_status() == (7, pkv.FLAG_BAD_BLOCK_ID)
    b.tables[:, 3] = -7
    b.run()
    assert pkv.device_status() == (7, pkv.FLAG_BAD_BLOCK_ID)
    b.tables = good
    b.ctx[1] = -1
    out = b.run()
    assert pkv.device_status() == (7, pkv.FLAG_BAD_CONTEXT)
    b.check(out)
    b.ctx[1] = 10 * 16 + 1  # a table row holds 10 blocks
    b.run()
    assert pkv.device_status() == (7, pkv.FLAG_BAD_CONTEXT)


def test_rows_behind_the_batch_and_repeats():
    """Bit for bit the same over repeated calls on a dirty workspace, and nothing written past the batch."""
    b = Batch([9, 3], [1600, 333], [1600 + 77 * i for i in range(9)] + [400, 300, 336], "bf16", 4, 4, 128)
    ws = b.workspace()
    buf = torch.full((b.B + 2,) + b.q.shape[1:], 5.0, dtype=torch.float32, device="cuda")
    first = b.run(workspace=ws, out=buf[1:-1]).clone()
    assert bool((buf[0] == 5.0).all()) and bool((buf[-1] == 5.0).all())
    b.check(first)
    for _ in range(5):
        assert torch.equal(b.run(workspace=ws), first)


def test_workspace_too_small():
    b = Batch([2], [64], [70, 80], "bf16", 4, 2, 128)
    with pytest.raises(pkv.KVError) as e:
        b.run(workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5
    with pytest.raises(ValueError):
        b.run(workspace=torch.zeros(1 << 26, dtype=torch.uint8))


def test_streams_and_captured_graphs():
    """On another stream, and replayed with other lengths, groups and queries; two graphs with workspaces of their own."""
    b = Batch([6, 6], [800, 1600], [800 + 50 * i for i in range(6)] + [1600 + 90 * i for i in range(6)], "bf16", 4, 4, 128)
    side = torch.cuda.Stream()
    ws, ws2 = b.workspace(), b.workspace()
    side.wait_stream(torch.cuda.current_stream())
    out = b.run(workspace=ws, stream=side)
    side.synchronize()
    b.check(out)
    graphs, outs = [], []
    for w in (ws, ws2):
        g = torch.cuda.CUDAGraph()
        o = torch.full(b.q.shape, float("nan"), dtype=torch.float32, device="cuda")
        with torch.cuda.graph(g):
            b.run(workspace=w, out=o)
        graphs.append(g)
        outs.append(o)
    b.q.normal_()
    b.ctx.sub_(torch.arange(12, dtype=torch.int32, device="cuda"))  # some fall below their prefix
    b.plens.copy_(torch.tensor([640, 1600], dtype=torch.int32))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    for o in outs:
        b.check(o)


def test_offsets_past_32_bits():
    """A cache whose K alone is over 4 GiB, the shared blocks at its end."""
    NB, Hkv, bs, D = 140000, 8, 16, 128
    b = Batch([3], [160], [170, 190, 200], "f16", 4, Hkv, D)
    n = b.kc.shape[0]
    kc = torch.empty((NB, Hkv, bs, D), dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    kc[-n:], vc[-n:] = b.kc, b.vc
    out = pkv.paged_shared_prefix_attention(b.q, kc, vc, torch.where(b.tables >= 0, b.tables + (NB - n), b.tables), b.ctx, b.starts,
                                            b.plens, b.scale, out_dtype=torch.float32)
    b.check(out)


def test_binding_refuses():
    b = Batch([2], [64], [70, 80], "bf16", 4, 2, 128)
    for name, bad in (("ctx", b.ctx.long()), ("ctx", b.ctx[:1]), ("starts", b.starts[:1]), ("plens", b.plens.float()),
                      ("tables", b.tables[:1]), ("q", b.q.half()), ("q", b.q.transpose(0, 1)), ("kc", b.kc[..., :64]),
                      ("starts", b.starts.cpu())):
        keep = getattr(b, name)
        setattr(b, name, bad)
        with pytest.raises((ValueError, pkv.KVError)):
            pkv.paged_shared_prefix_attention(b.q, b.kc, b.vc, b.tables, b.ctx, b.starts, b.plens, b.scale)
        setattr(b, name, keep)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_layer_of_a_decode_step(fp8):
    """append_rope and the attention that reads it, as a step runs them: prompts shared through the prefix pool."""
    Hq, Hkv, D, bs, B, P = 8, 2, 128, 16, 5, 96
    blocks = pkv.PrefixCachePool(256, bs)
    prompt = list(range(1000, 1000 + P))
    rows = [blocks.allocate(prompt + [7000 + 100 * i + t for t in range(20 + 9 * i)])[0] for i in range(B)]
    assert all(r[:P // bs] == rows[0][:P // bs] for r in rows)
    ctx = [P + 20 + 9 * i for i in range(B)]
    mb = max(len(r) for r in rows)
    tables = torch.tensor([r + [-1] * (mb - len(r)) for r in rows], dtype=torch.int32, device="cuda")
    lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    pool = pkv.KVPool(1, 256, bs, Hkv, D, E4M3 if fp8 else torch.bfloat16)
    pool.buffer.zero_()
    scales = dict(k_scale=KS, v_scale=VS) if fp8 else {}
    rope = pkv.Rope((1e4 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)))
    g = torch.Generator(device="cuda").manual_seed(3)
    # Prefill: the first sequence brings the whole prompt, the others what follows the shared blocks.
    for s in range(B):
        first = 0 if s == 0 else P
        n = ctx[s] - 1 - first
        qs = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        slots = pkv.slot_mapping_varlen(tables[s:s + 1], qs, lens[s:s + 1] - 1, bs, 256, num_tokens=n)
        kv = torch.randn((n, 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        pos = torch.arange(first, ctx[s] - 1, dtype=torch.int32, device="cuda")
        pool.append_rope(0, kv[:, :Hkv], kv[:, Hkv:], slots, pos, rope, **scales)
    # The decode step.
    qkv = torch.randn((B, Hq + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    slots = pkv.slot_mapping(tables, lens, bs, 256)
    q = pool.append_rope(0, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], slots, lens - 1, rope, q=qkv[:, :Hq], **scales)
    kc, vc = pool.layer(0)
    starts = torch.tensor([0, B], dtype=torch.int32, device="cuda")
    plens = torch.tensor([P], dtype=torch.int32, device="cuda")
    out = pkv.paged_shared_prefix_attention(q, kc, vc, tables, lens, starts, plens, D ** -0.5, out_dtype=torch.float32, **scales)
    assert pkv.device_status() == (0, 0)
    check = Batch.__new__(Batch)
    check.__dict__.update(q=q, kc=kc, vc=vc, tables=tables, ctx=lens, bs=bs, fp8=fp8, Hkv=Hkv, G=Hq // Hkv, D=D, scale=D ** -0.5)
    check.check(out, "step")
    same = pkv.paged_decode_attention(q, kc, vc, tables, lens, D ** -0.5, out_dtype=torch.float32, **scales)
    check.check(same, "plain decode")
