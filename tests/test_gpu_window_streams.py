"""GPU tests of the windowed attention on other streams, in replayed graphs whose queries change, and from several host
threads at once, each result against the formula in 64 bits.

Tolerance: that of test_gpu_window_attention.py."""
import threading

import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv
from test_gpu_window_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("new", [None, [30, 1, 200]])
@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("f16", True)])
def test_replays_follow_the_queries(new, dtype, fp8):
    b = Batch([400, 33, 200], 64, 4, new=new, dtype=dtype, fp8=fp8)
    ws, out = b.workspace(), torch.empty(b.q.shape, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.run(workspace=ws, out=out, stream=side)
    side.synchronize()
    b.check(out, "another stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(workspace=ws, out=out)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for i in range(3):
        b.q.copy_(torch.randn(b.q.shape, generator=gen, device="cuda"))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        b.check(out, f"replay {i}")


def test_threads_with_streams_of_their_own():
    """Calls whose shapes and launch sizes differ, started together, each with its own stream and workspace."""
    batches = [Batch([700, 90, 3], 300, 5, dtype="bf16", Hkv=4, seed=1), Batch([2000] * 40, 1000, 0, dtype="f16", Hkv=2, bs=64, seed=2),
               Batch([900, 64], 128, 4, new=[500, 64], dtype="bf16", seed=3), Batch([500] * 6, 100, 2, new=[33] * 6, dtype="f16", D=64, bs=32, seed=4),
               Batch([700, 90], 300, 5, dtype="bf16", fp8=True, seed=5), Batch([600, 300], 200, 0, new=[200, 300], dtype="f16", fp8=True, seed=6)]
    outs = [torch.empty((4, *b.q.shape), device="cuda") for b in batches]
    barrier, errors = threading.Barrier(len(batches)), []
    torch.cuda.synchronize()

    def calls(b, out):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                barrier.wait()
                for o in out:
                    b.run(out=o)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(repr(e))

    threads = [threading.Thread(target=calls, args=x) for x in zip(batches, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for b, out in zip(batches, outs):
        for o in out:
            b.check(o)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("G", [1, 4])
def test_query_rows_behind_the_last_sequence(G, value):
    """They may hold anything: no row of the batch changes, and those of out stay."""
    b = Batch([300, 90], 64, 4, new=[120, 7], dtype="bf16", G=G, pad=200)
    kept = b.run()
    b.q[127:] = value
    out = b.run()
    assert torch.equal(out, kept) and bool((out[127:] == 7).all())
    assert pkv.device_status() == (0, 0)
