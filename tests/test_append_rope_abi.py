"""CPU-only tests of kv_rope_create and kv_append_rope: what they refuse, and
that a refusal comes before any CUDA call (device addresses here are made up)."""
import ctypes
import math

import pytest

import paged_kv_cache_slots_gb300 as pkv

INVALID, UNSUPPORTED = 1, 2
F32, F16, BF16, E4M3 = 0, 1, 2, 3
BASE = 1 << 32  # made-up device addresses


@pytest.fixture(scope="module")
def lib():
    return pkv.load_library()


def _rope(lib, rot=64, interleaved=0, axes=1, amplitude=1.0, freq=None, axis=None, null_freq=False):
    n = max(1, rot // 2)
    freq = [1.0 / (i + 1) for i in range(n)] if freq is None else freq
    cfg = pkv._RopeConfig(rot, interleaved, axes, amplitude, None if null_freq else (ctypes.c_double * len(freq))(*freq),
                          None if axis is None else (ctypes.c_int32 * len(axis))(*axis))
    h = ctypes.c_void_p()
    return lib.kv_rope_create(ctypes.byref(cfg), ctypes.byref(h)), h


def _pool(lib, dtype=BF16, kv_heads=2, head_dim=64):
    cfg = pkv._PoolConfig(2, 8, 16, kv_heads, head_dim, dtype, 0)
    h = ctypes.c_void_p()
    assert lib.kv_pool_create(ctypes.byref(cfg), ctypes.c_void_p(BASE), lib.kv_pool_bytes(ctypes.byref(cfg)), ctypes.byref(h)) == 0
    return h


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), INVALID), (dict(rot=63), INVALID), (dict(rot=-2), INVALID), (dict(rot=258), UNSUPPORTED),
    (dict(axes=0), INVALID), (dict(axes=9), INVALID), (dict(amplitude=math.inf), INVALID), (dict(amplitude=math.nan), INVALID),
    (dict(null_freq=True), INVALID), (dict(rot=4, freq=[1.0, math.nan]), INVALID), (dict(rot=4, freq=[math.inf, 1.0]), INVALID),
    (dict(rot=4, axes=2, axis=[0, 2]), INVALID), (dict(rot=4, axes=2, axis=[-1, 0]), INVALID),
    (dict(rot=2), 0), (dict(rot=256), 0), (dict(rot=4, axes=8, axis=[7, 0]), 0), (dict(rot=4, freq=[-1.0, 1e30]), 0)])
def test_rope_create(lib, kw, status):
    st, h = _rope(lib, **kw)
    assert st == status
    assert (h.value is not None) == (status == 0)
    lib.kv_rope_destroy(h)


def test_rope_create_null(lib):
    assert lib.kv_rope_create(None, None) == INVALID
    lib.kv_rope_destroy(None)


def _call(lib, pool, rope, **kw):
    d = dict(layer=0, seq_ids=None, n=4, k=BASE + (1 << 24), k_stride=128, v=BASE + (2 << 24), v_stride=128, dtype=BF16,
             slots=BASE + (3 << 24), pos=BASE + (4 << 24), pos_stride=4, q=BASE + (5 << 24), q_stride=256,
             q_out=BASE + (6 << 24), q_out_stride=256, heads=4, ks=1.0, vs=1.0)
    d.update(kw)
    P = ctypes.c_void_p
    return lib.kv_append_rope(pool, d["layer"], rope, P(d["seq_ids"]), d["n"], P(d["k"]), d["k_stride"], P(d["v"]), d["v_stride"],
                              d["dtype"], P(d["slots"]), P(d["pos"]), d["pos_stride"], P(d["q"]), d["q_stride"], P(d["q_out"]),
                              d["q_out_stride"], d["heads"], d["ks"], d["vs"], None)


Q = BASE + (5 << 24)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(layer=2), INVALID), (dict(layer=-1), INVALID), (dict(dtype=F16), INVALID), (dict(dtype=E4M3), INVALID),
    (dict(dtype=7), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(pos=None), INVALID),
    (dict(q_out=None), INVALID), (dict(heads=0), INVALID), (dict(heads=-1), INVALID), (dict(k_stride=127), INVALID),
    (dict(v_stride=127), INVALID), (dict(q_stride=255), INVALID), (dict(q_out_stride=255), INVALID), (dict(k=BASE + 1), INVALID),
    (dict(q=Q + 1), INVALID), (dict(pos=BASE + 2), INVALID), (dict(seq_ids=BASE + 2), INVALID),
    # q_out over q other than in place, over k, over v
    (dict(q_out=Q + 2), INVALID), (dict(q_out=Q, q_out_stride=512), INVALID), (dict(q_out=Q + 512 * 3), INVALID),
    (dict(q_out=BASE + (1 << 24) + 64), INVALID), (dict(q_out=BASE + (2 << 24) - 8), INVALID)])
def test_append_rope_refuses(lib, kw, status):
    pool, (st, rope) = _pool(lib), _rope(lib)
    assert st == 0
    assert _call(lib, pool, rope, **kw) == status
    assert lib.kv_last_error()
    lib.kv_rope_destroy(rope)
    lib.kv_pool_destroy(pool)


def test_append_rope_refuses_null_handles_and_wide_rotation(lib):
    pool, (_, rope) = _pool(lib), _rope(lib)
    assert _call(lib, None, rope) == INVALID
    assert _call(lib, pool, None) == INVALID
    _, wide = _rope(lib, rot=128)
    assert _call(lib, pool, wide) == INVALID  # heads of 64
    _, axes = _rope(lib, rot=64, axes=3, axis=[i % 3 for i in range(32)])
    assert _call(lib, pool, axes, pos_stride=3) == INVALID
    for h in (rope, wide, axes):
        lib.kv_rope_destroy(h)
    lib.kv_pool_destroy(pool)


@pytest.mark.parametrize("ks,vs", [(0.0, 1.0), (1.0, -1.0), (math.inf, 1.0), (1.0, math.nan)])
def test_append_rope_refuses_bad_scales(lib, ks, vs):
    pool, (_, rope) = _pool(lib, dtype=E4M3), _rope(lib)
    assert _call(lib, pool, rope, ks=ks, vs=vs) == INVALID
    lib.kv_rope_destroy(rope)
    lib.kv_pool_destroy(pool)


def test_no_tokens_is_a_no_op(lib):
    pool, (_, rope) = _pool(lib), _rope(lib)
    assert _call(lib, pool, rope, n=0, k=None, v=None, slots=None, pos=None, q=None, q_out=None) == 0
    lib.kv_rope_destroy(rope)
    lib.kv_pool_destroy(pool)


def test_binding_refuses_bad_ropes():
    with pytest.raises(ValueError):
        pkv.Rope([])
    with pytest.raises(ValueError):
        pkv.Rope([1.0, 0.5], axes=[0])
    with pytest.raises(pkv.KVError):
        pkv.Rope([1.0, math.nan])
    with pytest.raises(pkv.KVError):
        pkv.Rope([1.0, 0.5], axes=[0, -1])
    r = pkv.Rope([1.0, 0.5], axes=[1, 0])
    assert (r.rot_dim, r.num_axes) == (4, 2)
