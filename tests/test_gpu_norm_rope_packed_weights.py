"""GPU test of norm weights that stand in one buffer with q_out, between its tokens' rows or next to them: as if they stood
elsewhere, bit for bit; where they reach into a row the call is refused and nothing is written."""
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("tokens", [1, 5, 700, 5000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weights_beside_the_rows(tokens, dtype):
    Hq, Hkv, D, bs = 8, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(tokens)
    q, k, v = (torch.randn((tokens, h, D), generator=g, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv))
    slots = torch.randperm(tokens, generator=g, device="cuda").int()
    positions = torch.arange(tokens, dtype=torch.int32, device="cuda")
    rope = pkv.Rope(10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D))
    w = (1 + 0.1 * torch.randn((2, D), generator=g, device="cuda")).to(dtype)

    def run(qw, kw, out):
        pool = pkv.KVPool(1, -(-tokens // bs), bs, Hkv, D, dtype, device="cuda")
        pool.buffer.zero_()  # (slots that no token is written to would differ by chance)
        pool.append_norm_rope(0, k, v, slots, positions, rope, kw, q=q, q_weight=qw, q_out=out)
        torch.cuda.synchronize()
        return out.clone(), pool.buffer.clone()

    want = run(w[0].clone(), w[1].clone(), torch.empty_like(q))
    row = Hq * D + 2 * D
    packed = torch.zeros(tokens * row + D, dtype=dtype, device="cuda")
    out = packed[:tokens * row].view(tokens, row)[:, :Hq * D].view(tokens, Hq, D)
    gap = packed[(tokens - 1) * row + Hq * D:][:2 * D].view(2, D)  # behind the last row, and between rows:
    first = packed[Hq * D:][:2 * D].view(2, D)
    for place in (gap, first):
        place.copy_(w)
        got = run(place[0], place[1], out)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(place, w)
    kept = packed.clone()
    for start in (Hq * D - 16, (tokens - 1) * row, row + Hq * D - D // 2 if tokens > 1 else 0):
        with pytest.raises(pkv.KVError):
            run(packed[start:][:D], w[1], out)
    assert torch.equal(packed, kept)
    assert pkv.device_status() == (0, 0)
