"""GPU test of the shared-prefix attention where one key outweighs each of thousands of others some 2^25 times, and the
others make up the whole output.

Tolerance: that of test_gpu_shared_prefix.py, and what the two f16 parts of a weight lose below their smallest step.
The weights enter them 2^7 times as large as (at most) the largest, so each loses at most 2^-25 * 2^-7 of the largest
weight, n of them n * 2^-32 * max |v| of the output."""
import math

import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv
from test_gpu_shared_prefix import DT, KS, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype,D,fp8", [("f16", 64, False), ("f16", 128, False), ("bf16", 64, False), ("f16", 128, True),
                                         ("bf16", 128, True)])
@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("apart", [25.5, 28.0])
def test_many_small_weights(dtype, D, fp8, place, apart):
    n, Hkv = 8192, 32
    b = Batch([2], [n], [n, n], dtype, 1, Hkv, D, fp8=fp8)
    one = 44.0 if fp8 else 1.0
    b.kc.copy_(torch.zeros(b.kc.shape, device="cuda"))
    b.vc.copy_(torch.full(b.vc.shape, one, device="cuda"))
    key = {"first": 0, "middle": n // 2 + 5, "last": n - 1}[place]
    blk = b.tables[0, key // 16].long()
    view = torch.uint8 if fp8 else b.kc.dtype
    row = torch.zeros(D, device="cuda")
    row[0] = 56.0 if fp8 else 1.0
    b.kc.view(view)[blk, :, key % 16] = row.to(b.kc.dtype).view(view)
    b.vc.view(view)[blk, :, key % 16] = torch.zeros(D, device="cuda").to(b.vc.dtype).view(view)
    b.q.zero_()
    b.q[:, :, 0] = apart / math.log2(math.e)
    b.scale = 1.0
    out = b.run()
    ref, tol = b.expected()
    assert float(ref.min()) > 2.0 ** -17
    off = (out.double() - ref).abs() - tol - n * 2.0 ** -32
    assert float(off.max()) <= 0, f"{float(off.max()):.3e} past the bound, of {float(ref.max()):.3e}"
    assert KS == 1 / 56 and DT[dtype] == b.q.dtype


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [30.0, 300.0, 1000.0, 2500.0])
@pytest.mark.parametrize("order", ["rising", "falling", "any"])
def test_scores_of_any_size(dtype, size, order):
    """Scores up to 10^8, steps between them of whole units and more: the weights stay in f16's range, and the output is a
    mean of V's rows, within their bounds but for the rounding of the weights' sum and the product's (2^-10 in all)."""
    n = 3000
    b = Batch([3], [n], [n, n + 7, n + 40], dtype, 2, 4, 128, seed=int(size))
    b.q.copy_(b.q.sign() * size)
    along = torch.linspace(-1, 1, n // 16, device="cuda")
    if order == "any":
        along = along[torch.randperm(n // 16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))]
    if order == "falling":
        along = -along
    unit = b.q[0].float().view(4, 2, 128)[:, 0].sign()  # along the first query of each KV head
    blk = b.tables[0, :n // 16].long()
    noise = torch.nan_to_num(b.kc[blk].float()) * 0.01
    b.kc[blk] = ((along.view(-1, 1, 1, 1) + noise) * unit.view(1, 4, 1, 128) * size).to(b.kc.dtype)
    out = b.run()
    assert pkv.device_status() == (0, 0)
    assert torch.isfinite(out).all()
    for s, c in enumerate(b.ctx.tolist()):
        v = b.vc[b.tables[s, :-(-c // 16)].long()].double().transpose(0, 1).flatten(1, 2)[:, :c]  # [KV, c, D]
        lo, hi = (x.repeat_interleave(2, 0) for x in (v.amin(1), v.amax(1)))
        slack = 2.0 ** -10 * v.abs().amax(1).repeat_interleave(2, 0)
        assert bool((out[s].double() >= lo - slack).all()) and bool((out[s].double() <= hi + slack).all())
