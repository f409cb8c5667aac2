"""GPU tests of the normalising, rotating append (KVPool.append_norm_rope) against the formula in 64 bits.

Tolerance.  The sum of squares adds positive fp32 terms, at most D / 4 + 8 roundings on
the way of one of them (a lane's elements, and five steps over the lanes): off by that
many 2^-24 relatively; the mean and eps add two more.  Its reciprocal root halves that
and is off by 2^-22 itself; times the weight and the element, two roundings more.  So z is
within (D / 8 + 4 + 1 + 4 + 2 + 1) 2^-24 of itself; the rotation of z is then held to the
bounds of the rotating append.
"""
import pytest
import torch

import oracle
import paged_kv_cache_slots_gb300 as pkv
import test_gpu_append_rope as plain

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Case(plain.Case):
    """weights: "same" (the rows' type) or "f32"; per_head: a row of weights for each head; None: no weights."""

    def __init__(self, *args, weights="same", per_head=False, eps=1e-6, spread=1.0, wshift=0, **kw):
        super().__init__(*args, **kw)
        g = torch.Generator().manual_seed(5)
        self.eps, dt = eps, self.q.dtype
        if spread != 1.0:  # rows of very different sizes
            f = spread ** (torch.rand((self.q.shape[0], 1, 1), generator=g) * 2 - 1).cuda()
            self.q.copy_((self.q.float() * f).to(dt))
            self.k.copy_((self.k.float() * f).to(dt))
        self.w = []
        for x in (self.q, self.k):
            shape = x.shape[1:] if per_head else x.shape[2:]
            w = (1 + 0.3 * torch.randn(shape, generator=g)).to(torch.float32 if weights == "f32" else dt)
            buf = torch.empty(w.numel() + wshift, dtype=w.dtype, device="cuda")
            buf[wshift:] = w.reshape(-1).cuda()
            self.w.append(None if weights is None else buf[wshift:].view(shape))

    def run(self, **kw):
        return self.pool.append_norm_rope(1, self.k, self.v, self.slots, self.pos, self.rope, self.w[1], q=self.q, q_weight=self.w[0],
                                          eps=self.eps, **self.scales, **kw)

    def rows(self, x, w):
        """(y, bound before rounding) of rows x in float64."""
        z = x.double().cpu()
        D = z.shape[-1]
        z = z / (z.square().mean(-1, keepdim=True) + self.eps).sqrt()
        if w is not None:
            z = z * w.double().cpu()
        y, e = plain.formula(z, self.pos, self.freq, self.axis, self.inter, self.amp)
        n, rho = len(self.freq), (D / 8 + 12) * 2.0 ** -24
        ia = torch.arange(0, 2 * n, 2) if self.inter else torch.arange(n)
        ib = ia + 1 if self.inter else ia + n
        off = z.abs() * rho
        both = (off[..., ia] + off[..., ib]) * abs(self.amp) * (1 + 2.0 ** -20)
        off[..., ia] = off[..., ib] = both
        return y, e + off

    def check(self, q_out, seq_ids=None):
        assert pkv.device_status() == (0, 0)
        T, bs = self.slots.shape[0], self.bs
        live = torch.ones(T, dtype=torch.bool) if seq_ids is None else seq_ids.cpu() >= 0
        slots = self.slots.cpu().long()
        put = live & (slots >= 0)
        if q_out is not None:
            y, e = self.rows(self.q, self.w[0])
            plain.near(q_out[live.cuda()], y[live], e[live], "q")
        kc, vc = (c.view(torch.uint8).cpu() for c in self.pool.layer(1))
        k0, v0 = (c.view(torch.uint8) for c in self.pool.layer(0))
        assert bool((k0 == 0x2B).all()) and bool((v0 == 0x2B).all())
        blk, off = slots[put] // bs, slots[put] % bs
        rest = torch.ones(kc.shape[:1] + kc.shape[2:3], dtype=torch.bool)
        rest[blk, off] = False
        for c in (kc, vc):
            assert bool((c.transpose(1, 2)[rest] == 0x2B).all()), "a slot that no token names was written"
        y, e = self.rows(self.k, self.w[1])
        y, e = y[put], e[put]
        krows, vrows = kc[blk, :, off], vc[blk, :, off]
        if self.fp8:
            want = y / self.scales["k_scale"]
            slack = e / self.scales["k_scale"] + want.abs() * 2.0 ** -23
            half = torch.maximum(want.abs() * 2.0 ** -4, torch.full_like(want, 2.0 ** -10))
            got = krows.contiguous().view(E4M3).double()
            assert bool(((got - want.clamp(-448, 448)).abs() <= half + slack).all())
            codes = oracle.quantize_e4m3(self.v.float().cpu()[put].contiguous(), self.scales["v_scale"])
            assert torch.equal(vrows, codes.view(torch.uint8))
        else:
            plain.near(krows.contiguous().view(self.k.dtype), y, e, "k")
            assert torch.equal(vrows.contiguous().view(self.v.dtype), self.v.cpu()[put])


SHAPES = plain.SHAPES + [
    (1, 32, 8, 128, 128, "bf16", dict(weights="f32")),
    (130, 8, 2, 128, 128, "f16", dict(weights="f32", per_head=True)),
    (130, 8, 2, 128, 64, "bf16", dict(per_head=True, packed=True)),
    (70, 6, 3, 80, 20, "f16", dict(weights="f32", interleaved=True, bs=7)),
    (70, 6, 3, 80, 20, "f32", dict(per_head=True)),
    (50, 4, 2, 128, 128, "bf16", dict(wshift=1)),
    (50, 4, 2, 128, 128, "bf16", dict(weights="f32", wshift=1)),
    (50, 4, 2, 128, 128, "bf16", dict(wshift=4, per_head=True)),
    (50, 4, 2, 128, 128, "bf16", dict(weights=None)),
    (64, 4, 2, 128, 128, "bf16", dict(spread=1e4)),
    (64, 4, 2, 96, 32, "f32", dict(spread=1e6, eps=0.0)),
    (64, 4, 2, 64, 64, "f16", dict(spread=1e-3, eps=1e-5)),
    # many tokens of whole 16-byte items
    (333, 7, 3, 128, 128, "f16", dict(packed=True, interleaved=True)),
    (700, 5, 2, 96, 32, "f16", dict(packed=True, axes=3)),
    (2100, 16, 2, 128, 64, "bf16", dict(weights="f32", per_head=True, packed=True)),
    (701, 8, 8, 64, 64, "f32", dict(per_head=True, amplitude=1.5)),
    (400, 3, 1, 256, 256, "bf16", dict(weights=None, interleaved=True)),
    (400, 2, 1, 512, 128, "f16", {}),
    (320, 122, 8, 128, 128, "bf16", dict(packed=True)),
    (320, 123, 8, 128, 128, "bf16", dict(packed=True)),
    (9, 2, 1, 1040, 16, "f16", {}),
    (9, 3, 1, 1032, 6, "bf16", dict(weights="f32", per_head=True)),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,kw", SHAPES, ids=lambda x: str(x) if not isinstance(x, dict) else "_".join(x))
def test_against_the_formula(T, Hq, Hkv, D, rot, dtype, kw):
    c = Case(T, Hq, Hkv, D, rot, dtype, **kw)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,kw", [
    (1, 8, 2, 128, 128, {}), (130, 8, 2, 128, 64, dict(interleaved=True, packed=True)), (45, 2, 3, 80, 20, dict(bs=8)),
    (900, 6, 3, 128, 64, dict(packed=True, weights="f32")), (310, 4, 2, 64, 64, dict(interleaved=True)),
    (45, 2, 1, 48, 2, dict(interleaved=True, weights="f32")), (20, 1, 2, 16, 16, dict(shift=1)), (6, 1, 1, 1040, 2, {})])
def test_quantized(T, Hq, Hkv, D, rot, dtype, kw):
    c = Case(T, Hq, Hkv, D, rot, dtype, fp8=True, **kw)
    c.check(c.run())


@pytest.mark.parametrize("T,D", [(40, 64), (40, 1040), (650, 128)])
@pytest.mark.parametrize("fp8", [False, True])
def test_negative_slots_and_padding(fp8, T, D):
    c = Case(T, 8, 2, D, 64, "bf16", fp8=fp8)
    c.slots[3] = c.slots[17] = -1
    c.slots[18] = -(2 ** 31)
    ids = torch.arange(T, dtype=torch.int32, device="cuda")
    ids[5] = ids[39] = -1
    q_out = torch.full_like(c.q, 7.0)
    assert c.run(q_out=q_out, seq_ids=ids) is q_out
    c.check(q_out, ids)
    assert bool((q_out[[5, 39]] == 7.0).all())
    fresh = c.run(seq_ids=ids)
    assert bool((fresh[[5, 39]] == 0).all())


@pytest.mark.parametrize("T", [12, 400])
def test_slots_past_the_pool_are_flagged(T):
    c = Case(T, 4, 2, 64, 64, "f16")
    n = c.NB * c.bs
    c.slots[2], c.slots[7] = n, 2 ** 31 - 1
    q_out = c.run()
    assert pkv.device_status() == (7, pkv.FLAG_BAD_SLOT)
    c.slots[2] = c.slots[7] = -1
    c.check(q_out)


@pytest.mark.parametrize("T,D", [(77, 128), (77, 1040), (1200, 128)])
@pytest.mark.parametrize("inter", [False, True])
def test_in_place_and_without_q(inter, T, D):
    c = Case(T, 8, 2, D, 128, "bf16", packed=True, interleaved=inter)
    want = c.run()
    before = c.q.clone()
    got = c.run(q_out=c.q)
    assert got is c.q and torch.equal(got, want)
    c.q.copy_(before)
    c.check(want)
    c.pool.buffer.fill_(0x2B)
    assert c.pool.append_norm_rope(1, c.k, c.v, c.slots, c.pos, c.rope, c.w[1], eps=c.eps) is None
    c.check(want)


@pytest.mark.parametrize("T", [30, 500])
def test_rows_are_apart(T):
    """Zero rows, and rows with an infinity or a NaN, leave the others alone."""
    c = Case(T, 8, 2, 128, 128, "bf16")
    want = c.run()
    c.q[3, 1] = 0
    c.q[4, 2, 5] = float("inf")
    c.q[5, 3, 77] = float("nan")
    got = c.run()
    same = torch.ones((T, 8), dtype=torch.bool, device="cuda")
    same[3, 1] = same[4, 2] = same[5, 3] = False
    assert torch.equal(got[same], want[same])
    assert bool((got[3, 1] == 0).all())
    assert bool(got[5, 3].isnan().all())


def test_captured_and_on_another_stream():
    c = Case(200, 16, 4, 128, 128, "bf16", packed=True, axes=3)
    want = c.run()
    c.check(want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(q_out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    side = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    c.run(q_out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)


def test_refuses_wrong_weights():
    c = Case(6, 4, 2, 64, 64, "bf16")
    kw, qw = c.w[1], c.w[0]

    def call(k_weight=kw, q_weight=qw, **more):
        return c.pool.append_norm_rope(1, c.k, c.v, c.slots, c.pos, c.rope, k_weight, **{"q": c.q, "q_weight": q_weight, **more})

    call()
    for bad in (kw.half(), kw[:32], kw.cpu(), kw[None].expand(3, 64).contiguous(), torch.empty(128, dtype=kw.dtype, device="cuda")[::2],
                kw.double()):
        with pytest.raises(ValueError):
            call(k_weight=bad)
    with pytest.raises(ValueError):
        call(q_weight=qw.float())  # of another type than k_weight
    with pytest.raises(ValueError):
        call(q=None)
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(pkv.KVError):
            call(eps=eps)
