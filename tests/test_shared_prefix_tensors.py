"""CPU-only tests of the tensors that paged_shared_prefix_attention's binding refuses: none of these calls reaches the
library, whose kernels would take a host address for a device one."""
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv

I32 = torch.int32


def _args(dtype=torch.bfloat16):
    return dict(q=torch.zeros((2, 8, 128), dtype=dtype), k_cache=torch.zeros((4, 2, 16, 128), dtype=dtype),
                v_cache=torch.zeros((4, 2, 16, 128), dtype=dtype), block_tables=torch.zeros((2, 3), dtype=I32),
                context_lens=torch.ones(2, dtype=I32), group_start=torch.tensor([0, 2], dtype=I32),
                prefix_lens=torch.tensor([16], dtype=I32), scale=0.1, out=torch.zeros((2, 8, 128), dtype=dtype),
                workspace=torch.zeros(1 << 20, dtype=torch.uint8), stream=0)


@pytest.fixture
def no_library_call(monkeypatch):
    def call(*_):
        raise AssertionError("the library was called")

    monkeypatch.setattr(pkv, "_call_on", call)


@pytest.mark.parametrize("leave_out", [(), ("out",), ("workspace",), ("out", "workspace"), ("stream",),
                                       ("stream", "out", "workspace")])
def test_host_tensors(no_library_call, leave_out):
    args = {k: v for k, v in _args().items() if k not in leave_out}
    with pytest.raises(ValueError, match="GPU"):
        pkv.paged_shared_prefix_attention(**args)


def test_host_tensors_of_an_e4m3_cache(no_library_call):
    args = _args()
    args.update(k_cache=args["k_cache"].to(torch.float8_e4m3fn), v_cache=args["v_cache"].to(torch.float8_e4m3fn), k_scale=1.0,
                v_scale=1.0)
    with pytest.raises(ValueError, match="GPU"):
        pkv.paged_shared_prefix_attention(**args)


class _OnGpu(torch.Tensor):
    """A host tensor that says it is on GPU 0."""

    def get_device(self):
        return 0


def test_a_workspace_with_gaps(no_library_call):
    args = {k: v.as_subclass(_OnGpu) if isinstance(v, torch.Tensor) else v for k, v in _args().items()}
    for bad in (torch.zeros(1 << 20, dtype=torch.uint8)[::2], torch.zeros((1, 8), dtype=torch.uint8).expand(1 << 18, 8)):
        args["workspace"] = bad.as_subclass(_OnGpu)
        with pytest.raises(ValueError, match="workspace"):
            pkv.paged_shared_prefix_attention(**args)
    args["workspace"] = torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(_OnGpu)
    with pytest.raises(AssertionError, match="library"):  # these are in order
        pkv.paged_shared_prefix_attention(**args)


@pytest.mark.parametrize("name", ["k_cache", "v_cache", "block_tables", "context_lens", "group_start", "prefix_lens", "out",
                                  "workspace"])
def test_one_tensor_on_the_host(no_library_call, name):
    args = {k: v.as_subclass(_OnGpu) if isinstance(v, torch.Tensor) and k != name else v for k, v in _args().items()}
    with pytest.raises(ValueError, match="GPU"):
        pkv.paged_shared_prefix_attention(**args)
