"""GPU tests of the ways in which positions lie for a rope with several axes."""
import pytest
import torch

from test_gpu_append_rope import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("T", [1, 2, 37, 700])
@pytest.mark.parametrize("axes", [2, 3, 8])
def test_one_row_expanded_to_all_axes(T, axes):
    """Text tokens of a model with several axes: the same position on each."""
    c = Case(T, 8, 2, 128, 128, "bf16", axes=axes)
    c.pos = c.pos[:1].expand(axes, T)
    assert c.pos.stride(0) == 0 or T == 1
    c.check(c.run())


@pytest.mark.parametrize("T", [1, 5])
def test_one_position_for_all(T):
    c = Case(T, 4, 2, 64, 64, "f16", axes=3)
    c.pos = torch.tensor(41, dtype=torch.int32, device="cuda").expand(3, T)
    c.check(c.run())


@pytest.mark.parametrize("T", [1, 64])
def test_columns_and_slices(T):
    c = Case(T, 4, 2, 64, 64, "f16", axes=3)
    base = c.pos.t().contiguous()  # [tokens, axes]
    keep = c.pos
    for pos in (base.t(), torch.cat((keep, keep), 1)[:, T:], torch.stack((keep, keep), 2)[..., 1]):
        c.pos = pos
        c.pool.buffer.fill_(0x2B)
        got = c.run()
        c.pos = keep
        c.check(got)


def test_one_axis_as_a_row():
    c = Case(9, 4, 2, 64, 64, "bf16")
    row = c.pos
    for pos in (row, row[0], row[:, :1].expand(1, 9) * 0 + row, torch.stack((row[0], row[0]), 1)[:, 0]):
        c.pos = pos
        c.pool.buffer.fill_(0x2B)
        got = c.run()
        c.pos = row
        c.check(got)
