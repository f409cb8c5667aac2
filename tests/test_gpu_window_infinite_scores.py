"""GPU tests of the windowed attention where some keys in sight have scores of -inf: their weights are 0, wherever they
stand and however many, and the others make up the row.  A row whose keys all have such scores is NaN, as the formula is.

Tolerance: that of test_gpu_window_attention.py."""
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv
from test_gpu_window_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def expected(b, s, gone):
    """(out, bound) of sequence s in float64, keys at positions `gone` (a mask) left out."""
    n, c = b.new[s], b.ctx_list[s]
    at = slice(s, s + 1) if b.decode else slice(b.start_list[s], b.start_list[s] + n)
    p, j = torch.arange(c - n, c, device="cuda")[:, None], torch.arange(c, device="cuda")
    seen = (j <= p) & ((j > p - b.window) | (j < b.sinks)) & ~gone
    k, v = (torch.where(seen.any(0)[None, :, None], torch.nan_to_num(b.rows(s, x, 1)), 0.0) for x in (b.kc, b.vc))
    q = b.q[at].double().view(n, b.Hkv, b.G, b.D).permute(1, 2, 0, 3)
    w = torch.softmax((q @ k[:, None].mT * b.scale).masked_fill(~seen, -torch.inf), -1)
    err = b.D * 2.0 ** -24 * b.scale * (q.abs() @ k[:, None].abs().mT).amax(-1, keepdim=True)
    bound = w @ v[:, None].abs() * (4 * err + 2.0 ** -15 + 2 * c * 2.0 ** -24)
    return at, *((x.permute(2, 0, 1, 3).reshape(n, -1, b.D)) for x in (w @ v[:, None], bound))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [None, [70, 5]])
@pytest.mark.parametrize("first,last", [(0, 20), (700, 740), (800, 870), (830, 835), (0, 880)])
def test_keys_of_minus_infinity(dtype, D, new, first, last):
    for G, opts in ((4, {}), (8, {}), (1, {}), *([(4, dict(consumer_warps=8)), (4, dict(separate_reduce=True))] if new is None else [])):
        b = Batch([900, 40], 210, 20, new=new, dtype=dtype, G=G, D=D, seed=G)
        b.q[..., 0] = b.q[..., 0].abs() + 0.5
        at = torch.arange(first, last, device="cuda")
        blk = b.tables[0].long()[at // b.bs]
        at, blk = at[blk >= 0], blk[blk >= 0]
        b.kc[blk, :, at % b.bs, 0] = -torch.inf
        gone = torch.zeros(900, dtype=torch.bool, device="cuda")
        gone[first:last] = True
        out = b.run(**opts).double()
        assert pkv.device_status() == (0, 0)
        for s, mask in ((0, gone), (1, torch.zeros(40, dtype=torch.bool, device="cuda"))):
            rows, ref, bound = expected(b, s, mask)
            none = ref.isnan()  # a row that sees no other key
            assert torch.equal(out[rows].isnan(), none), (G, opts, s)
            assert bool(((out[rows] - ref).abs() <= bound)[~none].all()), (G, opts, s)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("new", [None, [70, 5]])
def test_nothing_but_minus_infinity(dtype, new):
    b = Batch([300, 40], 100, 3, new=new, dtype=dtype)
    b.q[..., 0] = b.q[..., 0].abs() + 0.5
    b.kc[b.tables[0][b.tables[0] >= 0].long(), :, :, 0] = -torch.inf
    out = b.run()
    rows = 1 if new is None else 70
    assert bool(out[:rows].isnan().all()) and torch.isfinite(out[rows:]).all()
    assert pkv.device_status() == (0, 0)
