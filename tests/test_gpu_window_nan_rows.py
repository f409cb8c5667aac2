"""GPU tests of chunks under a window in which rows have to be computed again because a V element that some rows see is no
number: rows of many items of one CTA, and rows over so many keys that they take longer than any wait in the kernel may.

Tolerance: that of test_gpu_window_attention.py."""
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv
from test_gpu_window_attention import DT, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,D,G", [("bf16", 128, 4), ("f16", 64, 8), ("f16", 128, 1)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_rows_of_many_items(dtype, D, G, value):
    window, n = 300, 2500
    b = Batch([2600, 2000], window, 3, new=[n, 700], dtype=dtype, G=G, Hkv=8, D=D, pad=2)
    clean, bound = b.expected()
    part = b.part
    sees = torch.zeros(b.q.shape, dtype=torch.bool, device="cuda")
    for s, at, h, d in ((0, 1, 2, 7), (0, 1500, 2, 0), (0, 1777, 7, D - 1), (1, 1990, 0, 33), (0, 2599, 5, 1)):
        b.vc[int(b.tables[s, at // b.bs]), h, at % b.bs, d] = value
        p = torch.arange(b.ctx_list[s] - b.new[s], b.ctx_list[s], device="cuda")
        rows = b.start_list[s] + ((at <= p) & ((at > p - window) | (at < 3))).nonzero()[:, 0]
        sees[rows, h * G:(h + 1) * G, d] = True
    for dt in (torch.float32, DT[dtype]):
        out = b.run(dt)
        assert pkv.device_status() == (0, 0)
        tol = bound if dt == torch.float32 else bound + part + torch.finfo(dt).eps / 2 * (clean.abs() + bound) + torch.finfo(dt).smallest_normal
        assert not torch.isfinite(out[sees]).any()
        off = torch.where(sees, -1.0, (out.double() - clean).abs() - tol)
        assert bool((off <= 0).all()), f"{float(off.max()):.3e} past the bound"


def test_rows_that_take_seconds():
    """128 rows of the first item over 262,144 keys, 32 of them one after another in each of four warps (some 2.4 s),
    while the CTA has another item to do."""
    n, window, G, D = 9800, 262144, 4, 128
    ctx = window + n
    b = Batch([ctx], window, 0, new=[n], dtype="bf16", G=G, Hkv=1, D=D, bs=32)
    at = 32  # positions 32 .. : the first 32 tokens see it
    b.vc[int(b.tables[0, at // b.bs]), 0, at % b.bs, 5] = float("nan")
    out = b.run().double()
    assert pkv.device_status() == (0, 0)
    k, v = b.rows(0, b.kc, 1)[0], b.rows(0, b.vc, 1)[0]
    v[at, 5] = 0.0
    for t in (0, 1, 31, 32, 63, 64, 127, 152 * 64, 152 * 64 + 63, n - 1):
        p = window + t
        kk, vv = k[p - window + 1:p + 1], v[p - window + 1:p + 1]
        q = b.q[t].double()
        w = torch.softmax(q @ kk.T * b.scale, -1)
        err = D * 2.0 ** -24 * abs(b.scale) * (q.abs() @ kk.abs().T).amax(-1, keepdim=True)
        tol = w @ vv.abs() * (4 * err + 2.0 ** -15 + 2 * window * 2.0 ** -24)
        off = (out[t] - w @ vv).abs() - tol
        if t < 32:
            assert bool(out[t, :, 5].isnan().all())
            off[:, 5] = -1
        assert float(off.max()) <= 0, t
