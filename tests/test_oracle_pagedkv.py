"""Pins of the paged-cache oracle (oracle/pagedkv.py) on the CPU: hand-made
tables, the way back through the truncation, attention against torch's softmax
on dense keys."""

import numpy as np
import pytest
import torch

from oracle import blocktable, pagedkv


def test_extend_by_hand():
    # bs 4; sequence 0: 3 tokens + 2 -> one block; 1: 4 + 0 -> none; 2: 0 + 9 -> three
    table = np.array([[7, -1, -1], [8, -1, -1], [-1, -1, -1]])
    r = pagedkv.blocktable_extend(table, [3, 4, 0], [2, 0, 9], [10, 11, 12, 13, 14, 0], 5, 4, 13)
    assert r["block_table"].tolist() == [[7, 14, -1], [8, -1, -1], [13, 12, 11]]
    assert r["new_lens"].tolist() == [5, 4, 9] and r["num_taken"].tolist() == [1, 0, 3]
    assert r["free_left"] == 1 and r["cu_tokens"].tolist() == [0, 2, 2, 11]
    assert r["slot_map"].tolist() == [31, 56, 52, 53, 54, 55, 48, 49, 50, 51, 44, -1, -1]
    assert r["positions"].tolist() == [3, 4, 0, 1, 2, 3, 4, 5, 6, 7, 8, -1, -1]


def test_extend_refusals_leave_the_sequence():
    table = np.full((5, 2), -1)
    r = pagedkv.blocktable_extend(table, [0, 0, -1, 0, 0], [-3, 9, 1, 5, 0], [1, 2, 3], 1, 4, 100)
    # negative n; beyond the table; negative L; two blocks needed, one there; nothing needed
    assert r["num_taken"].tolist() == [-1, -1, -1, -2, 0]
    assert r["new_lens"].tolist() == [0, 0, -1, 0, 0] and (r["block_table"] == -1).all()
    assert r["cu_tokens"].tolist() == [0, 0, 9, 10, 15, 15] and r["free_left"] == 1
    assert (r["slot_map"] == -1).all()


def test_extend_undoes_truncate():
    rng = np.random.default_rng(3)
    B, bs = 9, 5
    lens = rng.integers(1, 40, B)
    table = np.full((B, 9), -1)
    ids = iter(rng.permutation(200))
    for b in range(B):
        for i in range(-(-int(lens[b]) // bs)):
            table[b, i] = next(ids)
    drop = np.array([int(rng.integers(0, min(12, n) + 1)) for n in lens])
    t2, l2, freed, nf = blocktable.kv_blocktable_truncate(table, lens, drop, bs, 4)
    r = pagedkv.blocktable_extend(t2, l2, drop, np.full(50, -1), 0, bs, int(drop.sum()), freed, nf)
    assert (r["new_lens"] == lens).all() and r["free_left"] == 0
    assert sorted(r["block_table"].ravel()) == sorted(table.ravel())
    assert ((r["block_table"] >= 0) == (table >= 0)).all()


def test_append_puts_rows_at_their_slots():
    cache = np.zeros((3, 2, 4, 5))
    rows = np.arange(40, dtype=np.float64).reshape(4, 2, 5)
    out = pagedkv.cache_append(rows, [5, -1, 12, 11], cache)
    assert (out[1, :, 1] == rows[0]).all() and (out[2, :, 3] == rows[3]).all()
    # rows 1 and 2 (past the cache) went nowhere: 2 x 10 values, the first of which is 0
    assert np.count_nonzero(out) == 19


@pytest.mark.parametrize("window", [0, 5])
def test_attention_against_dense_softmax(window):
    g = torch.Generator().manual_seed(1)
    H, kv, D, bs, L, n = 6, 2, 8, 4, 19, 7
    table = np.array([[4, 0, 3, 1, 2]])
    kc = torch.randn((5, kv, bs, D), generator=g, dtype=torch.float64)
    vc = torch.randn((5, kv, bs, D), generator=g, dtype=torch.float64)
    q = torch.randn((n + 2, H, D), generator=g, dtype=torch.float64)
    r = pagedkv.paged_attention(q.numpy(), kc.numpy(), vc.numpy(), table, [L], [1, 1 + n], 0.3,
                                window)
    k = kc[table[0]].transpose(1, 2).reshape(-1, kv, D)[:L].repeat_interleave(H // kv, 1)
    v = vc[table[0]].transpose(1, 2).reshape(-1, kv, D)[:L].repeat_interleave(H // kv, 1)
    pos = torch.arange(L - n, L)[:, None]
    key = torch.arange(L)
    ok = (key <= pos) & ((key > pos - window) if window else True)
    x = torch.einsum("qhd,khd->hqk", q[1:1 + n], k) * 0.3
    x = x.masked_fill(~ok, float("-inf"))
    ref = torch.einsum("hqk,khd->qhd", torch.softmax(x, -1), v)
    assert np.abs(r["out"][1:1 + n] - ref.numpy()).max() < 1e-12
    assert np.abs(r["lse"][1:1 + n] - torch.logsumexp(x, -1).T.numpy()).max() < 1e-12
    assert np.isnan(r["out"][0]).all() and np.isnan(r["out"][-1]).all()


def test_attention_rows_that_see_nothing():
    z = np.ones((2, 1, 4, 8))
    # three rows of a sequence of length 2 (the first before position 0), a page off the cache
    r = pagedkv.paged_attention(np.ones((4, 1, 8)), z, z, np.array([[0], [-1]]), [2, 1], [0, 3, 4], 1.0)
    assert (r["out"][0] == 0).all() and r["lse"][0] == -np.inf
    assert (r["out"][1:3] == 1).all() and (r["out"][3] == 0).all() and r["lse"][3, 0] == -np.inf
