"""CPU-only tests of what the windowed attention calls, kv_append_norm_rope and the kv_tables calls refuse: each
refusal comes before any CUDA call (device addresses here are made up)."""
import ctypes
import math

import pytest

import paged_kv_cache_slots_gb300 as pkv
from test_append_rope_abi import _pool, _rope

INVALID, UNSUPPORTED, TOO_SMALL = 1, 2, 5
F32, F16, BF16, E4M3 = 0, 1, 2, 3
A = 1 << 32  # a made-up device address
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    return pkv.load_library()


def _decode(lib, fp8=False, **kw):
    d = dict(q=A, k=A, v=A, NB=64, tables=A, mb=16, ctx=A, B=4, Hq=8, Hkv=2, D=128, bs=16, dtype=BF16, scale=0.1, window=100,
             sinks=4, out=A, out_dtype=BF16, ws=A, ws_bytes=1 << 40, ks=1.0, vs=1.0)
    d.update(kw)
    sizes = (d["NB"], P(d["tables"]), d["mb"], P(d["ctx"]), d["B"], d["Hq"], d["Hkv"], d["D"], d["bs"])
    end = (d["scale"], d["window"], d["sinks"], P(d["out"]), d["out_dtype"], P(d["ws"]), d["ws_bytes"], None, None)
    if fp8:
        return lib.paged_window_decode_attention_fp8(P(d["q"]), d["dtype"], P(d["k"]), P(d["v"]), d["ks"], d["vs"], *sizes, *end)
    return lib.paged_window_decode_attention(P(d["q"]), P(d["k"]), P(d["v"]), *sizes, d["dtype"], *end)


def _prefill(lib, fp8=False, **kw):
    d = dict(q=A, k=A, v=A, NB=64, tables=A, mb=16, start=A, ctx=A, B=4, T=9, Hq=8, Hkv=2, D=128, bs=16, dtype=BF16, scale=0.1,
             window=100, sinks=4, out=A, out_dtype=BF16, ws=A, ws_bytes=1 << 40, ks=1.0, vs=1.0)
    d.update(kw)
    sizes = (d["NB"], P(d["tables"]), d["mb"], P(d["start"]), P(d["ctx"]), d["B"], d["T"], d["Hq"], d["Hkv"], d["D"], d["bs"])
    end = (d["scale"], d["window"], d["sinks"], P(d["out"]), d["out_dtype"], P(d["ws"]), d["ws_bytes"], None)
    if fp8:
        return lib.paged_window_prefill_attention_fp8(P(d["q"]), d["dtype"], P(d["k"]), P(d["v"]), d["ks"], d["vs"], *sizes, *end)
    return lib.paged_window_prefill_attention(P(d["q"]), P(d["k"]), P(d["v"]), *sizes, d["dtype"], *end)


BOTH = [
    (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(mb=1 << 27), UNSUPPORTED),
    (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=9), INVALID), (dict(NB=0), INVALID),
    (dict(mb=0), INVALID), (dict(Hq=6), UNSUPPORTED), (dict(Hq=32), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(bs=512), UNSUPPORTED), (dict(out_dtype=F16), UNSUPPORTED), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(NB=1 << 27), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(tables=None), INVALID), (dict(ctx=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
    (dict(q=A + 8), INVALID), (dict(k=A + 8), INVALID), (dict(out=A + 4), INVALID), (dict(dtype=9), INVALID)]


@pytest.mark.parametrize("kw,status", BOTH + [(dict(ws=A + 128), INVALID)])
def test_decode_refuses(lib, kw, status):
    assert _decode(lib, **kw) == status
    assert lib.kv_last_error()


@pytest.mark.parametrize("kw,status", BOTH + [(dict(bs=24), UNSUPPORTED), (dict(bs=8), UNSUPPORTED), (dict(T=-1), INVALID),
                                              (dict(start=None), INVALID), (dict(dtype=E4M3), INVALID), (dict(ws=A + 8), INVALID)])
def test_prefill_refuses(lib, kw, status):
    assert _prefill(lib, **kw) == status
    assert lib.kv_last_error()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [dict(out=A), dict(out=A + 9 * 8 * 128 * 2 - 16), dict(out=A - 16),
                                dict(out=A - 9 * 8 * 128 * 4 + 16, out_dtype=F32)])
def test_prefill_refuses_out_over_q(lib, fp8, kw):
    assert _prefill(lib, fp8, **kw) == INVALID
    assert b"overlaps" in lib.kv_last_error()


@pytest.mark.parametrize("call", [_decode, _prefill])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F32), UNSUPPORTED), (dict(dtype=E4M3), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(ks=0.0), INVALID),
    (dict(vs=-1.0), INVALID), (dict(ks=math.inf), INVALID), (dict(vs=math.nan), INVALID), (dict(out_dtype=F16), UNSUPPORTED),
    (dict(window=0), INVALID), (dict(sinks=-2), INVALID)])
def test_fp8_refuses(lib, call, kw, status):
    got = call(lib, fp8=True, **kw)
    assert got == status or (kw == dict(dtype=E4M3) and got == INVALID)


def test_nothing_to_do(lib):
    none = dict(q=None, k=None, v=None, tables=None, ctx=None, out=None, ws=None)
    assert _decode(lib, B=0, **none) == 0
    assert _prefill(lib, B=0, start=None, **none) == 0
    assert _prefill(lib, T=0, start=None, **none) == 0


def test_prefill_workspace(lib):
    n = ctypes.c_size_t()
    f = lib.paged_window_prefill_workspace_bytes
    assert f(4, 100, 8, 2, 128, 0, None) == INVALID
    for bad in ((-1, 1, 8, 2, 128), (1, -1, 8, 2, 128), (1, 1, 0, 2, 128), (1, 1, 8, 0, 128), (1, 1, 9, 2, 128), (1, 1, 8, 2, 0)):
        assert f(*bad, 0, ctypes.byref(n)) == INVALID


def _norm(lib, pool, rope, **kw):
    d = dict(layer=0, seq_ids=None, n=4, k=A + (1 << 24), k_stride=128, v=A + (2 << 24), v_stride=128, dtype=BF16, slots=A + (3 << 24),
             pos=A + (4 << 24), pos_stride=4, q=A + (5 << 24), q_stride=256, q_out=A + (6 << 24), q_out_stride=256, heads=4,
             qw=A + (7 << 24), qws=0, kw=A + (8 << 24), kws=0, wt=BF16, eps=1e-6, ks=1.0, vs=1.0)
    d.update(kw)
    return lib.kv_append_norm_rope(pool, d["layer"], rope, P(d["seq_ids"]), d["n"], P(d["k"]), d["k_stride"], P(d["v"]), d["v_stride"],
                                   d["dtype"], P(d["slots"]), P(d["pos"]), d["pos_stride"], P(d["q"]), d["q_stride"], P(d["q_out"]),
                                   d["q_out_stride"], d["heads"], P(d["qw"]), d["qws"], P(d["kw"]), d["kws"], d["wt"], d["eps"],
                                   d["ks"], d["vs"], None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(layer=2), dict(dtype=F16), dict(dtype=7), dict(k=None), dict(v=None), dict(slots=None), dict(pos=None),
    dict(q_out=None), dict(heads=0), dict(k_stride=127), dict(q_stride=255), dict(k=A + 1), dict(q_out=A + (1 << 24) + 64),
    dict(wt=F16), dict(wt=E4M3), dict(wt=9), dict(eps=-1e-9), dict(eps=math.nan), dict(eps=math.inf), dict(kw=A + 1), dict(qw=A + 1),
    dict(qws=63), dict(kws=-64), dict(kw=A + 2, wt=F32)])
def test_norm_rope_refuses(lib, kw):
    pool, (st, rope) = _pool(lib), _rope(lib)
    assert st == 0
    assert _norm(lib, pool, rope, **kw) == INVALID
    assert lib.kv_last_error()
    assert _norm(lib, None, rope) == INVALID and _norm(lib, pool, None) == INVALID
    assert _norm(lib, pool, rope, n=0, k=None, v=None, slots=None, pos=None, q=None, q_out=None, qw=None, kw=None) == 0
    lib.kv_rope_destroy(rope)
    lib.kv_pool_destroy(pool)


def _extend(lib, **kw):
    d = dict(tables=A, mb=8, held=A + (1 << 20), new=A + (2 << 20), B=4, bs=16, NB=64, queue=A + (3 << 20), state=A + (4 << 20), T=10,
             ctx=A + (5 << 20), start=A + (6 << 20), slots=A + (7 << 20), pos=A + (8 << 20), seqs=A + (9 << 20), out=A + (10 << 20))
    d.update(kw)
    return lib.kv_tables_extend(P(d["tables"]), d["mb"], P(d["held"]), P(d["new"]), d["B"], d["bs"], d["NB"], P(d["queue"]), P(d["state"]),
                                d["T"], P(d["ctx"]), P(d["start"]), P(d["slots"]), P(d["pos"]), P(d["seqs"]), P(d["out"]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(mb=0), INVALID), (dict(bs=0), INVALID), (dict(NB=0), INVALID), (dict(T=-1), INVALID),
    (dict(B=8193), UNSUPPORTED), (dict(NB=1 << 27), UNSUPPORTED), (dict(mb=1 << 27), UNSUPPORTED),
    *[({x: None}, INVALID) for x in ("tables", "held", "new", "queue", "state", "ctx", "start", "slots", "pos", "seqs", "out")],
    *[({x: A + (11 << 20) + 2}, INVALID) for x in ("tables", "held", "new", "queue", "state", "ctx", "start", "slots", "pos", "seqs", "out")],
    # overlaps: two outputs; an output and an input that it is not the update of, or not in its place
    (dict(pos=A + (7 << 20) + 36), INVALID), (dict(start=A + 124), INVALID), (dict(ctx=A + (2 << 20)), INVALID),
    (dict(ctx=A + (1 << 20) + 4), INVALID), (dict(out=A + (3 << 20) + 252), INVALID), (dict(out=A + (4 << 20) + 4), INVALID),
    (dict(queue=A + 8), INVALID), (dict(seqs=A + (4 << 20)), INVALID)])
def test_extend_refuses(lib, kw, status):
    assert _extend(lib, **kw) == status
    assert lib.kv_last_error()


def _release(lib, **kw):
    d = dict(tables=A, mb=8, ctx=A + (1 << 20), B=4, bs=16, NB=64, done=A + (2 << 20), window=0, sinks=0, queue=A + (3 << 20),
             state=A + (4 << 20))
    d.update(kw)
    return lib.kv_tables_release(P(d["tables"]), d["mb"], P(d["ctx"]), d["B"], d["bs"], d["NB"], P(d["done"]), d["window"], d["sinks"],
                                 P(d["queue"]), P(d["state"]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(mb=0), INVALID), (dict(bs=0), INVALID), (dict(NB=0), INVALID), (dict(B=8193), UNSUPPORTED),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(tables=None), INVALID), (dict(ctx=None), INVALID),
    (dict(queue=None), INVALID), (dict(state=None), INVALID), (dict(done=A + 1), INVALID), (dict(done=A + (1 << 20) + 12), INVALID),
    (dict(queue=A + 120), INVALID)])
def test_release_refuses(lib, kw, status):
    assert _release(lib, **kw) == status
    assert lib.kv_last_error()


def test_release_of_no_sequences(lib):
    assert _release(lib, B=0, tables=None, ctx=None, done=None, queue=None, state=None) == 0


def test_binding_refuses_host_tensors():
    import torch

    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.extend_tables(z.view(2, 2), z[:2], z[:2], z, z[:2], 4, 4, out=pkv.StepTables(z[:2], torch.zeros(3, dtype=torch.int32), z, z, z, z[:2]))
    with pytest.raises(ValueError):
        pkv.release_tables(z.view(2, 2), z[:2], z, z[:2], 4)
    q, c = torch.zeros((2, 4, 128)), torch.zeros((3, 2, 16, 128))
    t = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.paged_window_decode_attention(q, c, c, t, z[:2], 1.0, 8)
    with pytest.raises(ValueError):
        pkv.paged_window_prefill_attention(q, c, c, t, z[:3], z[:2], 1.0, 8)
    with pytest.raises(ValueError):
        pkv.make_free_queue(1, reserve_null_block=True, device="cpu")
    assert pkv.make_free_queue(3, True, device="cpu")[0].tolist() == [1, 2, -1]
