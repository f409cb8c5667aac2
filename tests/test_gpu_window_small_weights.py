"""GPU tests of the windowed attention where one key outweighs each of thousands of others by up to 2^28, and the others
make up the whole output: what a first token that every query looks at, and whose V is near zero, does to a window.

Tolerance: that of test_gpu_window_attention.py, and what f16 parts of a weight lose below their smallest step, 2^-24.
The largest weight in sight of a row enters them as 2^15 (single tokens) or as 2^7 at least (chunks), so a weight loses at
most 2^-25 / 2^15 or 2^-25 / 2^7 of the largest one, n of them n * 2^-40 or n * 2^-32 of max |v| of the output.  bf16 parts
keep fp32's exponents and lose nothing more."""
import math

import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv
from test_gpu_window_attention import DT, Batch

pytestmark = pytest.mark.gpu
FORMS = [("f16", 64, False), ("f16", 128, False), ("bf16", 64, False), ("f16", 128, True), ("bf16", 128, True)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def one_large_weight(key, apart, dtype, D, fp8, G, n=8192, window=4096, **kw):
    """Key `key` of the first sequence scores `apart` (in powers of two) above the others and holds V = 0, they V = 1."""
    b = Batch([n, 300], window, 4, dtype=dtype, G=G, Hkv=2, D=D, fp8=fp8, **kw)
    view = torch.uint8 if fp8 else b.kc.dtype
    zeros = torch.zeros(D, device="cuda").to(b.kc.dtype).view(view)
    b.kc.view(view).copy_(zeros.expand(b.kc.shape))
    b.vc.view(view).copy_(torch.full((D,), 44.0 if fp8 else 1.0, device="cuda").to(b.vc.dtype).view(view).expand(b.vc.shape))
    blk = b.tables[0, key // b.bs].long()
    row = torch.zeros(D, device="cuda")
    row[0] = 56.0 if fp8 else 1.0
    b.kc.view(view)[blk, :, key % b.bs] = row.to(b.kc.dtype).view(view)
    b.vc.view(view)[blk, :, key % b.bs] = zeros
    b.q.zero_()
    b.q[:, :, 0] = apart / math.log2(math.e)
    b.scale = 1.0
    return b


def check(b, out, floor):
    assert pkv.device_status() == (0, 0)
    ref, tol = b.expected()
    if out.dtype != torch.float32:
        tol = tol + (0 if b.decode else b.part) + torch.finfo(out.dtype).eps / 2 * ref.abs() + torch.finfo(out.dtype).smallest_normal
    off = (out.double() - ref).abs() - tol - max(b.ctx_list) * floor
    assert float(off.max()) <= 0, f"{float(off.max()):.3e} past the bound, where {float(ref[0].max()):.3e} is due"


@pytest.mark.parametrize("dtype,D,fp8", FORMS)
@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("apart", [15.0, 20.0, 25.5, 28.0])
def test_chunks(dtype, D, fp8, place, apart):
    n, new = 8192, 130
    # the chunk's rows all see it: a first token, one in the middle of the window, the first new token
    key = {"first": 1, "middle": n - 2000, "last": n - new}[place]
    floor = 0.0 if dtype == "bf16" else 2.0 ** -32
    for G in (1, 4):
        b = one_large_weight(key, apart, dtype, D, fp8, G, n, new=[new, 3])
        check(b, b.run(), floor)
        check(b, b.run(DT[dtype]), floor)


@pytest.mark.parametrize("dtype,D,fp8", FORMS)
@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("apart", [15.0, 20.0, 25.5, 28.0])
@pytest.mark.parametrize("opts", [{}, dict(consumer_warps=8)])
def test_single_tokens(dtype, D, fp8, place, apart, opts):
    n = 8192
    key = {"first": 1, "middle": n - 2000, "last": n - 1}[place]
    for G in (1, 4, 8):
        b = one_large_weight(key, apart, dtype, D, fp8, G, n)
        check(b, b.run(**opts), 0.0 if dtype == "bf16" and not fp8 else 2.0 ** -40)


@pytest.mark.parametrize("dtype,fp8", [("f16", False), ("bf16", False), ("f16", True), ("bf16", True)])
@pytest.mark.parametrize("size", [3.0, 30.0, 300.0])
@pytest.mark.parametrize("order", ["rising", "falling"])
@pytest.mark.parametrize("new", [None, [200, 7]])
def test_scores_of_any_size(dtype, fp8, size, order, new):
    """Scores up to 10^7 that rise or fall along the keys, by fractions of a unit or by thousands a step: the weights stay
    in f16's range, and the output is a mean of V's rows, but for the rounding of the weights and their sum (2^-8 in all)."""
    n = 3000
    b = Batch([n, 77], 1500, 5, new=new, dtype=dtype, G=4, Hkv=2, fp8=fp8, seed=int(size))
    b.q.copy_(b.q.sign() * size)
    unit = b.q[:1].float().sign().view(2, 4, 128)[:, 0]
    blk = b.tables[0, :-(-n // 16)].long()
    held = blk >= 0
    along = torch.linspace(-1, 1, len(blk), device="cuda") * (1 if order == "rising" else -1)
    keys = along[held].view(-1, 1, 1, 1) * unit.view(1, 2, 1, 128) * min(size, 200.0)
    b.kc.view(torch.uint8 if fp8 else b.kc.dtype)[blk[held]] = keys.expand(-1, 2, 16, 128).to(b.kc.dtype).view(torch.uint8 if fp8 else b.kc.dtype)
    values = torch.nan_to_num(b.rows(0, b.vc, 1 / 44 if fp8 else 1))
    out = b.run().double()
    assert pkv.device_status() == (0, 0) and torch.isfinite(out).all()
    rows = 1 if new is None else new[0]
    lo, hi = (x.repeat_interleave(4, 0) for x in (values.amin(1), values.amax(1)))  # [Hq, D]
    slack = 2.0 ** -8 * values.abs().amax(1).repeat_interleave(4, 0)
    assert bool((out[:rows] >= lo - slack).all()) and bool((out[:rows] <= hi + slack).all())
