"""GPU test of host threads that make their first calls with different sizes at the same time, in a process of its own."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import threading
import torch
import paged_kv_cache_slots_gb300 as pkv

# Block sizes, heads and batches whose launches differ in shared memory, and for each its inputs.
SHAPES = [(16, 8, 4), (32, 8, 300), (48, 2, 20), (64, 4, 1500), (128, 2, 7), (208, 1, 40)]
work = []
for i, (bs, Hkv, B) in enumerate(SHAPES):
    g = torch.Generator(device="cuda").manual_seed(i)
    NB = 3 * B + 4
    kc, vc = (torch.randn((NB, Hkv, bs, 128), generator=g, device="cuda").half() for _ in range(2))
    own = torch.arange(4, 4 + 2 * B, device="cuda", dtype=torch.int32).view(B, 2)
    tables = torch.cat((torch.arange(4, device="cuda", dtype=torch.int32).expand(B, 4), own), 1).contiguous()
    ctx = 4 * bs + 1 + torch.arange(B, device="cuda", dtype=torch.int32) % (2 * bs)
    q = torch.randn((B, 4 * Hkv, 128), generator=g, device="cuda").half()
    starts = torch.tensor([0, B], dtype=torch.int32, device="cuda")
    plens = torch.tensor([4 * bs], dtype=torch.int32, device="cuda")
    work.append((q, kc, vc, tables, ctx, starts, plens))
torch.cuda.synchronize()
barrier = threading.Barrier(len(work))
got, errors = [None] * len(work), []


def calls(i):
    q, kc, vc, tables, ctx, starts, plens = work[i]
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            barrier.wait()
            for _ in range(3):
                a = pkv.paged_shared_prefix_attention(q, kc, vc, tables, ctx, starts, plens, 0.09, out_dtype=torch.float32)
                b = pkv.paged_decode_attention(q, kc, vc, tables, ctx, 0.09, out_dtype=torch.float32)
            torch.cuda.current_stream().synchronize()
            got[i] = (a, b)
    except Exception as e:  # noqa: BLE001
        errors.append((SHAPES[i], repr(e)))


threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(work))]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, errors
assert pkv.device_status() == (0, 0)
for (q, kc, vc, tables, ctx, starts, plens), (a, b), (bs, Hkv, B) in zip(work, got, SHAPES):
    for s in range(0, B, max(1, B // 5)):
        c = int(ctx[s])
        k, v = (x[tables[s].long()].double().transpose(0, 1).flatten(1, 2)[:, :c] for x in (kc, vc))
        want = (torch.softmax(q[s].double().view(Hkv, 4, 128) @ k.mT * 0.09, -1) @ v).flatten(0, 1)
        # fp32 results over at most 1248 keys: scores below 16 are off by 2^-13 at most, weights by 2^-15 more.
        for x in (a, b):
            assert float((x[s].double() - want).abs().max()) < 4 * (2.0 ** -13 + 2.0 ** -15), (bs, s)
for q, kc, vc, tables, ctx, starts, plens in work:  # every size is still allowed
    pkv.paged_shared_prefix_attention(q, kc, vc, tables, ctx, starts, plens, 0.09)
    pkv.paged_decode_attention(q, kc, vc, tables, ctx, 0.09)
assert pkv.device_status() == (0, 0)
print("threads ok")
"""


def test_first_calls_from_several_threads():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout + r.stderr
