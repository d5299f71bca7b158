"""Limits of the paged-KV calls on the CPU: what a call may ask for and what is
refused before any launch."""

import pytest

from tests.test_kv_abi_cpu import _attend, _extend, _ws, kv, sv   # noqa: F401

NOTHING = dict(q=None, k=None, v=None, table=None, lens=None, cu=None, out=None)


@pytest.mark.parametrize("batch", [(1 << 16) + 1, 1 << 20, 1 << 24, 2 ** 31 - 1])
def test_attention_refuses_batches_that_would_not_end(sv, kv, batch):   # noqa: F811
    for kw in (dict(), dict(dtype=0), dict(tokens=batch // 16, head_dim=256), dict(tokens=0)):
        assert _attend(sv, kv, NOTHING, batch=batch, **kw) == 2
        assert b"batch" in sv.library().spec_verify_last_error()
        assert _ws(sv, kv, batch=batch, **kw) == 0


def test_attention_takes_the_largest_batch(sv, kv):   # noqa: F811
    # passes the descriptor's checks: refused for its pointers alone
    assert _attend(sv, kv, dict(q=None), batch=1 << 16, tokens=1 << 16) == 1
    assert b"q is NULL" in sv.library().spec_verify_last_error()
    assert _ws(sv, kv, batch=1 << 16, tokens=1 << 16, max_blocks=4096, num_blocks=8192) > 0


def test_extension_takes_larger_ones(sv):   # noqa: F811
    assert _extend(sv, batch=1 << 24, lens=None) == 1
    assert _extend(sv, batch=(1 << 24) + 1) == 2
