"""GPU tests of chunks over E4M3 caches with every finite code, at every place of a row and of a tile.

V: under a window of 1 a token sees itself alone, so its row of out is its V row.  Its one weight need not be a power of
two exactly (the reference is a rounded product, the exponent one more rounding), so it meets V rounded, where the sum
that it is divided by is not: by 2^-17 (two parts, an fp32 output), or half a step of q's type and as much for the 16-bit
output itself, and 2^-22 for quotient and exponential.  Zeros and signs are exact, and neighbouring codes are 2^-4 apart.
K: against the formula in 64 bits with all codes of one exponent at a time and a scale that makes their scores differ by
whole units, so that a code taken for its neighbour, or a subnormal one for 0, is far outside; tolerance that of
test_gpu_window_attention.py."""
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv
from test_gpu_window_attention import E4M3, KS, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def finite(codes):
    return torch.where((codes & 0x7F) == 0x7F, codes & 0x80, codes).to(torch.uint8)


def store(b, cache, codes):
    """codes [ctx, Hkv, D] of the batch's one sequence, into its blocks."""
    n = codes.shape[0]
    at = torch.arange(n, device="cuda")
    cache.view(torch.uint8)[b.tables[0].long()[at // b.bs], :, at % b.bs] = codes


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [16, 32, 48])
@pytest.mark.parametrize("out_dtype", [torch.float32, None])
def test_every_value(dtype, bs, out_dtype):
    n = 700
    b = Batch([n], 1, 0, new=[n], dtype=dtype, G=4, Hkv=2, bs=bs, fp8=True)
    t, h, d = torch.meshgrid(torch.arange(n, device="cuda"), torch.arange(2, device="cuda"), torch.arange(128, device="cuda"), indexing="ij")
    codes = finite((37 * t + 11 * d + 128 * h + (t >> 8)) & 0xFF)
    store(b, b.vc, codes)
    assert len(codes.unique()) == 254
    out = pkv.paged_window_prefill_attention(b.q, b.kc, b.vc, b.tables, b.start, b.ctx, b.scale, 1, out_dtype=out_dtype, k_scale=KS,
                                             v_scale=1.0)
    want = codes.view(E4M3).float().repeat_interleave(4, 1)
    near = 2.0 ** -16 if out_dtype else torch.finfo(b.q.dtype).eps + 2.0 ** -16
    assert bool(((out.float() - want).abs() <= near * want.abs()).all())
    assert torch.equal(out == 0, want == 0)
    assert pkv.device_status() == (0, 0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("exponent", range(16))
def test_every_key(dtype, exponent):
    n = 300
    b = Batch([n], 150, 2, new=[n], dtype=dtype, G=4, Hkv=2, fp8=True, seed=exponent)
    g = torch.Generator(device="cuda").manual_seed(exponent)
    low = torch.randint(0, 8, (n, 2, 128), generator=g, device="cuda")
    sign = torch.randint(0, 2, (n, 2, 128), generator=g, device="cuda") << 7
    store(b, b.kc, finite((exponent << 3) | low | sign))
    # values of about 2^(exponent - 7) (the subnormal ones of 2^-7), sums over 128 dims of some 11 times that
    b.scale = 2.0 ** (7 - max(exponent, 1)) / KS / 8
    b.check(b.run())
