"""kv_paged_attention_q4 at the last positions that a length of 32 bits can have, with a
sliding window (so that few pages are read, each held by many places of the table)."""

import numpy as np
import pytest
import torch

from tests import kvcases as C
from tests import kvq4cases as Q

pytestmark = pytest.mark.gpu

LAST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


def _run(sv, q, cache, table, lens, cu, window, **kw):
    on = dict(dtype=torch.int32, device=C.DEV)
    r = sv.kv_paged_attention_q4(q, cache, table, torch.tensor(lens, **on), torch.tensor(cu, **on),
                                 lse=True, sliding_window=window, **kw)
    torch.cuda.synchronize()
    return r["out"], r["lse"]


def _cache(sv, blocks, kv, bs, dim, seed):
    g = torch.Generator(device=C.DEV).manual_seed(seed)
    c = sv.make_kv_cache_q4(blocks, kv, bs, dim, device=C.DEV)
    for n in ("k_codes", "v_codes"):
        c[n].random_(0, 256, generator=g)
    c["k_scales"].fill_(125)
    c["v_scales"].uniform_(0.5, 1.5, generator=g)
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256, 96])
@pytest.mark.parametrize("new", [1, 9, 40])
def test_a_sequence_of_the_largest_length(sv, new, dim, dtype):
    """The same rows far from there and at the end, bit for bit."""
    bs, kv, heads, blocks, window = 1 << 18, 1, 2, 2, 300
    cache = _cache(sv, blocks, kv, bs, dim, dim)
    width = 2 ** 31 // bs
    table = torch.arange(width, dtype=torch.int32, device=C.DEV)[None] % blocks
    q = torch.randn((new, heads, dim), device=C.DEV, generator=torch.Generator(device=C.DEV).manual_seed(1)
                    ).to(C.DT[dtype])
    back = 1000 * bs                    # (a multiple of the table's turns)
    near = _run(sv, q, cache, table, [LAST - back], [0, new], window, max_new=new)
    far = _run(sv, q, cache, table, [LAST], [0, new], window, max_new=new)
    assert torch.equal(near[0], far[0]) and torch.equal(near[1], far[1])
    assert torch.isfinite(far[1]).all() and (far[0] != 0).any(-1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_behind_a_table_that_ends_there(sv, dim, dtype):
    """A table of 2^31 - 48 positions: rows whose window lies behind them see nothing,
    beside rows of the same tile that see some."""
    bs, columns, new, window = 5368709, 400, 30, 20
    cap = bs * columns
    assert cap == 2 ** 31 - 48
    cache = _cache(sv, 2, 1, bs, dim, 7)
    table = torch.arange(columns, dtype=torch.int32, device=C.DEV)[None] % 2
    q = torch.randn((new, 1, dim), device=C.DEV, generator=torch.Generator(device=C.DEV).manual_seed(2)
                    ).to(C.DT[dtype])
    out, lse = _run(sv, q, cache, table, [cap + 27], [0, new], window, max_new=new)
    pos = cap + 27 - new + np.arange(new)
    sees = torch.from_numpy(pos - window + 1 <= cap - 1)
    assert sees.sum() == 22
    assert (out.cpu()[~sees] == 0).all() and torch.isneginf(lse.cpu()[~sees]).all()
    assert torch.isfinite(lse.cpu()[sees]).all()
    # (and two pages of the table earlier)
    small = _run(sv, q, cache, table[:, :398], [cap + 27 - 2 * bs], [0, new], window, max_new=new)
    ref = Q.reference(dict(q=q.cpu(), cache={n: t[:, :, -64:].cpu() for n, t in cache.items()},
                           block_table=torch.tensor([[1]], dtype=torch.int32),
                           seq_lens=torch.tensor([64 + 27], dtype=torch.int32),
                           cu_tokens=torch.tensor([0, new], dtype=torch.int32)), None, window)
    for o, z in ((out, lse), small):
        Q.check(C.to64(o), C.to64(z), ref, dtype, dim)
