"""GPU tests of the rotating append (KVPool.append_rope) against the formula in 64 bits.

Tolerance.  The kernel's angle is off by at most 2^-32 turns (1.5e-9 rad) and
the conversion of the rest of a quarter turn to fp32 (pi/4 * 2^-25 rad); with
sincospif's last place (2^-24) a cosine or sine is off by less than 2^-23.
The two products and their sum add at most 2^-24 of each operand's and of the
result's size.  So y before its rounding is within
(|x_a| + |x_b|) * |A| * 2^-22 * 1.25 (the quarter for A's own rounding), and the
rounding to the row's type adds half a step of it, or of the smallest step.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_slots_gb300 as pkv

pytestmark = pytest.mark.gpu
T16 = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def angle(pos, f):
    """pos * f modulo 2 pi: the product and its remainder need more than 64-bit floats at far positions."""
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    t = pos.cpu().numpy().astype(np.longdouble) * np.longdouble(f)
    return torch.from_numpy(np.remainder(t, two_pi).astype(np.float64))


def formula(x, pos, freq, axis, interleaved, amplitude):
    """(y, bound before rounding) of rows x [T, H, D] in float64; pos [axes, T]."""
    n = len(freq)
    x = x.double().cpu()
    t = torch.stack([angle(pos[a], f) for a, f in zip(axis, freq)], 1)[:, None]  # [T, 1, n]
    ia = torch.arange(0, 2 * n, 2) if interleaved else torch.arange(n)
    ib = ia + 1 if interleaved else ia + n
    y, e = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = amplitude * (a * t.cos() - b * t.sin())
    y[..., ib] = amplitude * (b * t.cos() + a * t.sin())
    e[..., ia] = e[..., ib] = (a.abs() + b.abs()) * abs(amplitude) * 2.0 ** -22 * 1.25
    return y, e


def near(got, y, e, what):
    info = torch.finfo(got.dtype)
    half = info.eps / 2 * (y.abs() + e) + info.smallest_normal * info.eps / 2
    off = (got.double().cpu() - y).abs() - e - torch.where(e == 0, torch.zeros_like(half), half)
    assert float(off.max()) <= 0, f"{what}: off by {float(off.max()):.3e} past the bound"


class Case:
    def __init__(self, T, Hq, Hkv, D, rot, dtype, bs=16, interleaved=False, axes=1, packed=False, amplitude=1.0, far=5000,
                 fp8=False, seed=0, shift=0, NB=None):
        g = torch.Generator().manual_seed(seed + 1000 * T + D + rot)
        dt = T16[dtype]
        self.freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).tolist()
        self.axis = [(7 * i) % axes for i in range(rot // 2)]
        self.inter, self.amp, self.fp8, self.bs = interleaved, amplitude, fp8, bs
        rows = torch.randn((T, Hq + 2 * Hkv, D), generator=g).to(dt)
        if packed:
            base = rows.cuda()
            self.q, self.k, self.v = base[:, :Hq], base[:, Hq:Hq + Hkv], base[:, Hq + Hkv:]
        else:
            def own(x):  # `shift` elements into a buffer of its own
                buf = torch.empty(x.numel() + shift, dtype=dt, device="cuda")
                buf[shift:] = x.reshape(-1).cuda()
                return buf[shift:].view(x.shape)
            self.q, self.k, self.v = own(rows[:, :Hq]), own(rows[:, Hq:Hq + Hkv]), own(rows[:, Hq + Hkv:])
        NB = NB or -(-T // bs) + 3
        self.NB = NB
        self.slots = torch.randperm(NB * bs, generator=g)[:T].to(torch.int32).cuda()
        self.pos = torch.randint(-far, far + 1, (axes, T), generator=g).to(torch.int32).cuda()
        self.pool = pkv.KVPool(2, NB, bs, Hkv, D, E4M3 if fp8 else dt)
        self.pool.buffer.fill_(0x2B)  # a pattern, to see what is written
        self.rope = pkv.Rope(self.freq, interleaved=interleaved, axes=self.axis, amplitude=amplitude)
        self.scales = dict(k_scale=1 / 56, v_scale=1 / 44) if fp8 else {}

    def run(self, **kw):
        return self.pool.append_rope(1, self.k, self.v, self.slots, self.pos, self.rope, q=self.q, **self.scales, **kw)

    def check(self, q_out, seq_ids=None):
        """q_out and the whole of layer 1, and that layer 0 and the other slots are as they were."""
        assert pkv.device_status() == (0, 0)
        T, bs = self.slots.shape[0], self.bs
        live = torch.ones(T, dtype=torch.bool) if seq_ids is None else seq_ids.cpu() >= 0
        slots = self.slots.cpu().long()
        put = live & (slots >= 0)
        y, e = formula(self.q, self.pos, self.freq, self.axis, self.inter, self.amp)
        near(q_out[live.cuda()], y[live], e[live], "q")
        kc, vc = (c.view(torch.uint8).cpu() for c in self.pool.layer(1))
        k0, v0 = (c.view(torch.uint8) for c in self.pool.layer(0))
        assert bool((k0 == 0x2B).all()) and bool((v0 == 0x2B).all())
        blk, off = slots[put] // bs, slots[put] % bs
        rest = torch.ones(kc.shape[:1] + kc.shape[2:3], dtype=torch.bool)
        rest[blk, off] = False
        for c in (kc, vc):
            assert bool((c.transpose(1, 2)[rest] == 0x2B).all()), "a slot that no token names was written"
        y, e = formula(self.k, self.pos, self.freq, self.axis, self.inter, self.amp)
        y, e = y[put], e[put]
        krows, vrows = kc[blk, :, off], vc[blk, :, off]
        if self.fp8:
            # A code is within half a step of the quotient, whose own rounding is 2^-24 of it.
            want = y / self.scales["k_scale"]
            slack = e / self.scales["k_scale"] + want.abs() * 2.0 ** -23
            half = torch.maximum(want.abs() * 2.0 ** -4, torch.full_like(want, 2.0 ** -10))
            got = krows.contiguous().view(E4M3).double()
            assert bool(((got - want.clamp(-448, 448)).abs() <= half + slack).all())
            codes = oracle.quantize_e4m3(self.v.float().cpu()[put].contiguous(), self.scales["v_scale"])
            assert torch.equal(vrows, codes.view(torch.uint8))
        else:
            near(krows.contiguous().view(self.k.dtype), y, e, "k")
            assert torch.equal(vrows.contiguous().view(self.v.dtype), self.v.cpu()[put])


SHAPES = [
    # T, Hq, Hkv, D, rot, dtype, options
    (1, 32, 8, 128, 128, "bf16", {}),
    (1, 1, 1, 64, 64, "f16", dict(interleaved=True)),
    (3, 4, 2, 64, 32, "f32", dict(bs=1)),
    (33, 32, 8, 128, 128, "bf16", dict(packed=True)),
    (257, 8, 8, 128, 96, "f16", dict(packed=True, axes=3)),
    (100, 6, 3, 80, 20, "bf16", dict(interleaved=True, bs=7)),
    (31, 5, 1, 256, 256, "bf16", dict(axes=2, interleaved=True)),
    (31, 5, 1, 256, 2, "f16", {}),
    (17, 3, 3, 8, 2, "f16", {}),
    (17, 3, 1, 72, 36, "f32", dict(packed=True)),
    (700, 16, 2, 128, 64, "f32", dict(interleaved=True, axes=8)),
    (40, 2, 2, 1024, 128, "bf16", {}),
    (40, 2, 1, 520, 6, "f16", dict(interleaved=True)),
    (64, 4, 4, 128, 128, "bf16", dict(shift=1)),
    (64, 4, 4, 128, 128, "bf16", dict(shift=4, interleaved=True)),
    (64, 4, 4, 128, 128, "f32", dict(shift=2)),
    (50, 4, 2, 64, 64, "f16", dict(amplitude=1.3)),
    (50, 4, 2, 64, 64, "bf16", dict(amplitude=-0.5, interleaved=True)),
    (1500, 32, 8, 128, 128, "bf16", dict(packed=True, bs=32)),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,kw", SHAPES, ids=lambda x: str(x) if not isinstance(x, dict) else "_".join(x))
def test_against_the_formula(T, Hq, Hkv, D, rot, dtype, kw):
    c = Case(T, Hq, Hkv, D, rot, dtype, **kw)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,kw", [
    (1, 8, 2, 128, 128, {}), (130, 8, 2, 128, 64, dict(interleaved=True, packed=True)), (45, 2, 3, 80, 20, dict(bs=8)),
    (45, 2, 1, 48, 2, dict(interleaved=True)), (20, 1, 2, 16, 16, dict(shift=1))])
def test_quantized(T, Hq, Hkv, D, rot, dtype, kw):
    c = Case(T, Hq, Hkv, D, rot, dtype, fp8=True, **kw)
    c.check(c.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_negative_slots_and_padding(fp8):
    c = Case(40, 8, 2, 64, 64, "bf16", fp8=fp8)
    c.slots[3] = c.slots[17] = -1
    c.slots[18] = -(2 ** 31)
    ids = torch.arange(40, dtype=torch.int32, device="cuda")
    ids[5] = ids[39] = -1
    q_out = torch.full_like(c.q, 7.0)
    assert c.run(q_out=q_out, seq_ids=ids) is q_out
    c.check(q_out, ids)
    assert bool((q_out[[5, 39]] == 7.0).all())
    fresh = c.run(seq_ids=ids)
    assert bool((fresh[[5, 39]] == 0).all())


def test_slots_past_the_pool_are_flagged():
    c = Case(12, 4, 2, 64, 64, "f16")
    n = c.NB * c.bs
    c.slots[2], c.slots[7] = n, 2 ** 31 - 1
    q_out = c.run()
    assert pkv.device_status() == (7, pkv.FLAG_BAD_SLOT)
    c.slots[2] = c.slots[7] = -1
    c.check(q_out)


@pytest.mark.parametrize("inter", [False, True])
def test_in_place_and_without_q(inter):
    c = Case(77, 8, 2, 128, 128, "bf16", packed=True, interleaved=inter)
    want = c.run()
    before = c.q.clone()
    got = c.run(q_out=c.q)
    assert got is c.q and torch.equal(got, want)
    c.q.copy_(before)
    c.check(want)
    c.pool.buffer.fill_(0x2B)
    assert c.pool.append_rope(1, c.k, c.v, c.slots, c.pos, c.rope) is None
    c.check(want)


def test_extreme_positions():
    """Angles keep their precision at any int32 position."""
    c = Case(64, 2, 1, 128, 128, "f32")
    c.pos[0, :8] = torch.tensor([2 ** 31 - 1, -(2 ** 31), 0, 1, -1, 2 ** 30, 10 ** 6, -(10 ** 9)], dtype=torch.int32)
    c.check(c.run())


def test_padded_positions_and_strides():
    """Positions with a longer row stride, and rows with gaps between tokens."""
    c = Case(30, 4, 2, 64, 64, "bf16", axes=3)
    wide = torch.full((3, 64), 12345, dtype=torch.int32, device="cuda")
    wide[:, :30] = c.pos
    c.pos = wide[:, :30]
    buf = torch.full((30, 5, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf[:, 1:3] = c.k
    c.k = buf[:, 1:3]
    out = torch.full((30, 9, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    c.check(c.run(q_out=out[:, 2:6]))
    assert bool((out[:, :2] == 3.0).all()) and bool((out[:, 6:] == 3.0).all())


def test_nonfinite_rows_stay_in_their_pairs():
    c = Case(4, 2, 2, 64, 32, "f16")
    c.k[1, 0, 3] = float("inf")
    c.k[2, 1, 40] = float("nan")  # past the rotated part
    c.v[3, 0, 5] = float("nan")
    c.run()
    kc, vc = c.pool.layer(1)
    s = c.slots.cpu().long()
    bad_k = ~torch.isfinite(torch.stack([kc[x // 16, :, x % 16] for x in s]))
    want = torch.zeros_like(bad_k)
    want[1, 0, 3] = want[1, 0, 19] = want[2, 1, 40] = True
    assert torch.equal(bad_k, want)
    assert int(torch.isnan(torch.stack([vc[x // 16, :, x % 16] for x in s])).sum()) == 1


def test_offsets_past_32_bits():
    """The last blocks of a layer whose K alone is over 4 GiB."""
    Hkv, D, bs, NB = 8, 128, 16, 140000
    c = Case(5, 2, Hkv, D, 128, "f16", NB=1)
    c.pool = pkv.KVPool(1, NB, bs, Hkv, D, torch.float16)
    kc, vc = c.pool.layer(0)
    kc[-2:] = 1.0
    vc[-2:] = 1.0
    c.slots = torch.tensor([NB * bs - 1, NB * bs - 3, NB * bs - 17, NB * bs - 20, NB * bs - 32], dtype=torch.int32, device="cuda")
    c.pool.append_rope(0, c.k, c.v, c.slots, c.pos, c.rope, q=c.q)
    y, e = formula(c.k, c.pos, c.freq, c.axis, False, 1.0)
    s = c.slots.cpu().long()
    near(torch.stack([kc[x // bs, :, x % bs] for x in s]), y, e, "k")
    assert torch.equal(torch.stack([vc[x // bs, :, x % bs] for x in s]), c.v)
    assert int((vc[-2:] == 1.0).sum()) >= (32 - 5) * Hkv * D
    assert pkv.device_status() == (0, 0)


def test_another_stream_and_a_captured_graph():
    c = Case(19, 8, 2, 128, 128, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q_out = torch.zeros_like(c.q)
    c.run(q_out=q_out, stream=side)
    side.synchronize()
    c.check(q_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(q_out=q_out)
    # New inputs in the captured buffers; the handle's frequencies are part of the graph.
    c.q.normal_()
    c.k.normal_()
    c.pos.add_(17)
    c.slots.copy_(c.slots.flip(0))
    c.pool.buffer.fill_(0x2B)
    graph.replay()
    torch.cuda.synchronize()
    c.check(q_out)


def test_no_tokens():
    c = Case(1, 2, 1, 64, 64, "f16")
    e = torch.empty((0, 1, 64), dtype=torch.float16, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    c.pool.append_rope(0, e, e, i, i, c.rope)
    out = c.pool.append_rope(0, e, e, i, i, c.rope, q=torch.empty((0, 2, 64), dtype=torch.float16, device="cuda"))
    assert out.shape == (0, 2, 64)
    assert bool((c.pool.buffer == 0x2B).all())


def test_binding_refuses():
    c = Case(8, 4, 2, 64, 64, "bf16")
    call = lambda **kw: c.pool.append_rope(1, *[kw.get(n, getattr(c, n)) for n in ("k", "v", "slots", "pos", "rope")],
                                           q=kw.get("q", c.q), q_out=kw.get("q_out"), seq_ids=kw.get("seq_ids"))  # noqa: E731
    for bad in (dict(k=c.k.half()), dict(v=c.v.float()), dict(q=c.q.half()), dict(k=c.k[:, :1]), dict(k=c.k.transpose(1, 2)),
                dict(slots=c.slots.long()), dict(slots=c.slots[:5]), dict(pos=c.pos.long()), dict(pos=c.pos[:, :4]),
                dict(q_out=c.q[:, :2]), dict(q_out=torch.empty_like(c.q, dtype=torch.float32)), dict(k=c.k.cpu()),
                dict(seq_ids=c.slots.long()), dict(seq_ids=c.slots[:3]), dict(q=c.q[:4])):
        with pytest.raises(ValueError):
            call(**bad)
    flat = torch.zeros(c.q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.KVError):
        call(q=flat[:c.q.numel()].view(c.q.shape), q_out=flat[8:].view(c.q.shape))
    assert bool((c.pool.buffer == 0x2B).all())
