"""GPU test of the windowed decode with lengths far apart, one long sequence among short ones, and few heads under long
windows, with blocks of every size: on both sides of the rule that chooses between its two kernels, and each of them.

Tolerance: that of test_gpu_window_attention.py."""
import pytest
import torch

from test_gpu_window_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,bs,fp8", [("bf16", 16, False), ("f16", 64, False), ("bf16", 128, False), ("f16", 192, False),
                                          ("bf16", 32, True), ("f16", 128, True)])
@pytest.mark.parametrize("Hkv,window", [(1, 700), (1, 20000), (8, 3000), (8, 20000)])
def test_one_long_among_short_ones(dtype, bs, fp8, Hkv, window):
    short = [100 + i for i in range(11)] + [0, 1, 16]
    for ctx in ([21000], [21000, *short], [*short, 9000, 21000]):
        b = Batch(ctx, window, 3, dtype=dtype, Hkv=Hkv, bs=bs, fp8=fp8, seed=bs)
        b.check(b.run())
        b.check(b.run(consumer_warps=8))
