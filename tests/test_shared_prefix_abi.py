"""CPU-only tests of paged_shared_prefix_attention's refusals: each comes before
any CUDA call (device addresses here are made up)."""
import ctypes
import math

import pytest

import paged_kv_cache_slots_gb300 as pkv

INVALID, UNSUPPORTED = 1, 2
F32, F16, BF16, E4M3 = 0, 1, 2, 3
A = 1 << 32  # a made-up device address


@pytest.fixture(scope="module")
def lib():
    return pkv.load_library()


def _call(lib, fp8=False, **kw):
    d = dict(q=A, k=A, v=A, NB=64, tables=A, mb=16, ctx=A, B=4, starts=A, plens=A, ng=1, Hq=8, Hkv=2, D=128, bs=16,
             dtype=BF16, scale=0.1, out=A, out_dtype=BF16, ws=A, ws_bytes=1 << 40, ks=1.0, vs=1.0)
    d.update(kw)
    P = ctypes.c_void_p
    tail = (d["NB"], P(d["tables"]), d["mb"], P(d["ctx"]), d["B"], P(d["starts"]), P(d["plens"]), d["ng"], d["Hq"], d["Hkv"],
            d["D"], d["bs"])
    end = (d["scale"], P(d["out"]), d["out_dtype"], P(d["ws"]), d["ws_bytes"], None)
    if fp8:
        return lib.paged_shared_prefix_attention_fp8(P(d["q"]), d["dtype"], P(d["k"]), P(d["v"]), d["ks"], d["vs"], *tail, *end)
    return lib.paged_shared_prefix_attention(P(d["q"]), P(d["k"]), P(d["v"]), *tail, d["dtype"], *end)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(ng=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=9), INVALID),
    (dict(NB=0), INVALID), (dict(mb=0), INVALID), (dict(Hq=6), UNSUPPORTED), (dict(Hq=32), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(bs=8), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(bs=512), UNSUPPORTED), (dict(dtype=F32, out_dtype=F32), UNSUPPORTED),
    (dict(dtype=E4M3), INVALID), (dict(dtype=9), INVALID), (dict(out_dtype=F16), UNSUPPORTED), (dict(out_dtype=E4M3), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(mb=1 << 29), UNSUPPORTED), (dict(NB=1 << 27), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(tables=None), INVALID), (dict(ctx=None), INVALID),
    (dict(starts=None), INVALID), (dict(plens=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
    (dict(q=A + 8), INVALID), (dict(k=A + 8), INVALID), (dict(out=A + 4), INVALID), (dict(ws=A + 128), INVALID),
    (dict(starts=A + 2), INVALID), (dict(B=1 << 28), UNSUPPORTED)])
def test_refuses(lib, kw, status):
    assert _call(lib, **kw) == status
    assert lib.kv_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), UNSUPPORTED), (dict(dtype=E4M3), INVALID), (dict(D=64), UNSUPPORTED), (dict(ks=0.0), INVALID),
    (dict(vs=-1.0), INVALID), (dict(ks=math.inf), INVALID), (dict(vs=math.nan), INVALID), (dict(out_dtype=F16), UNSUPPORTED)])
def test_fp8_refuses(lib, kw, status):
    assert _call(lib, fp8=True, **kw) == status


def test_no_sequences_is_a_no_op(lib):
    assert _call(lib, B=0, ng=0, q=None, k=None, v=None, tables=None, ctx=None, starts=None, plens=None, out=None, ws=None) == 0


def test_workspace_arguments(lib):
    n = ctypes.c_size_t()
    assert lib.paged_shared_prefix_workspace_bytes(4, 1, 8, 2, 128, 0, None) == INVALID
    assert lib.paged_shared_prefix_workspace_bytes(4, 1, 9, 2, 128, 0, ctypes.byref(n)) == INVALID
    assert lib.paged_shared_prefix_workspace_bytes(-4, 1, 8, 2, 128, 0, ctypes.byref(n)) == INVALID
