"""GPU tests of the shared-prefix attention over an E4M3 cache where the score multiplier vanishes: a zero scale, and
query rows that are zero or far below the others.  Shared tokens that are no multiple of 64 leave masked scores in the
last key tile."""
import pytest
import torch

from test_gpu_shared_prefix import DT, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 128 ** -0.5, -0.1])
@pytest.mark.parametrize("plen", [112, 64 * 40 + 16])
def test_zero_scale_and_small_queries(dtype, scale, plen):
    b = Batch([5], [plen], [plen, plen + 1, plen + 40, plen + 200, plen + 16], dtype, 4, 2, 128, fp8=True)
    b.scale = scale
    b.q[0] = 0  # every head
    b.q[1, 3] = 0
    b.q[2, 0] *= 2.0 ** -20  # in f16 some elements become zero or subnormal
    if dtype == "bf16":
        b.q[3, 1] *= 2.0 ** -60
        b.q[3, 5] *= 2.0 ** -110
        b.q[4, 2] *= 2.0 ** 60  # with its scale this row is a maximum's value alone
        if scale:
            b.q[4, 2] = 0
    b.check(b.run(), "fp32")
    b.check(b.run(DT[dtype]), dtype)
