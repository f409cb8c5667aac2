"""CPU-only test of kv_append_norm_rope's refusal of weights that lie in what the call writes (device addresses here are
made up; each refusal comes before any CUDA call)."""
import pytest

import paged_kv_cache_slots_gb300 as pkv
from test_append_rope_abi import _pool, _rope
from test_window_step_abi import A, F32, INVALID, _norm

QO = A + (6 << 24)  # q_out: 4 tokens of 4 heads of 64, bf16: rows of 512 bytes, 512 apart unless said otherwise


@pytest.fixture(scope="module")
def lib():
    return pkv.load_library()


@pytest.mark.parametrize("kw", [
    dict(qw=QO), dict(kw=QO), dict(qw=QO + 2048 - 128), dict(qw=QO - 126), dict(kw=QO - 252, wt=F32), dict(kw=QO + 512 + 64),
    # a row for each head: only the last one's reaches q_out
    dict(qw=QO - 3 * 1024 - 126, qws=512), dict(kw=QO - 2 * 64 - 126, kws=64),
    # between the tokens' rows of a packed buffer, but too long for the gap, or starting in a row
    dict(q_out_stride=288, qw=QO + 512 + 2), dict(q_out_stride=512, qw=QO + 1024 - 126), dict(q_out_stride=512, qw=QO + 510),
    dict(n=1, q_out_stride=0, kw=QO + 384)])
def test_weights_in_q_out(lib, kw):
    pool, (st, rope) = _pool(lib), _rope(lib)
    assert st == 0
    assert _norm(lib, pool, rope, **kw) == INVALID
    assert b"overlaps the weights" in lib.kv_last_error()
    lib.kv_rope_destroy(rope)
    lib.kv_pool_destroy(pool)
