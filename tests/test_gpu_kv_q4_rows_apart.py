"""A row of kv_paged_attention_q4 has the same bits whatever the other rows of its tile
see: keys that only a later token or another head sees, however large their scores."""

import math

import pytest
import torch

from tests import kvcases as C
from tests import kvq4cases as Q

pytestmark = pytest.mark.gpu

SCALE = 1.0
NEW = 7
# Many sequences, so that a workgroup takes several units: whole sequences of two and
# three units, and splits of longer ones.
WHOLE = [180 + 16 * (b % 9) for b in range(450)]
SPLIT = [3000 + 16 * (b % 5) for b in range(48)]


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


def _case(heads, kv, dim, dtype, split, seed):
    """Sequences whose scores are about the same, but for one key of every unit after
    the first that every row sees: 2 units (2.9 in log2) above.  Queries have 1 in the
    last channel and 0 in the other channels of its group of 32, where keys hold
    what the tests set."""
    ctx = SPLIT if split else WHOLE
    g = torch.Generator().manual_seed(seed)
    lens = [c + NEW for c in ctx]
    need = [-(-L // 16) for L in lens]
    order = torch.randperm(sum(need), generator=g).to(torch.int32)
    table = torch.full((len(ctx), max(need)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        table[b, :n] = order[sum(need[:b]):sum(need[:b]) + n]
    rows = (sum(need), kv, 16)

    def codes():
        return torch.randint(0, 256, (*rows, dim // 2), generator=g, dtype=torch.uint8)
    cache = dict(k_codes=codes(), v_codes=codes(),
                 k_scales=torch.full((*rows, -(-dim // 128) * 4), 125, dtype=torch.uint8),
                 v_scales=torch.rand(rows, generator=g) + 0.5)
    cache["k_codes"][..., (dim - 32) // 2:] = 0
    cache["k_scales"][..., dim // 32 - 1] = 127
    q = torch.randn((NEW * len(ctx), heads, dim), generator=g) * (0.6 * dim ** -0.5)
    q[..., dim - 32:] = 0.0
    q[..., dim - 1] = 1.0
    case = dict(q=q.to(C.DT[dtype]), cache=cache, block_table=table,
                seq_lens=torch.tensor(lens, dtype=torch.int32),
                cu_tokens=torch.arange(0, q.shape[0] + 1, NEW, dtype=torch.int32))
    for b, L in enumerate(lens):
        for p in range(130, L - NEW, 128):
            _set(case, b, p, dim, 2.0)
    return case


def _set(case, b, pos, dim, score, head=slice(None), channel=None):
    """The key of a position scores ``score`` more against a query's 1 in ``channel``."""
    at = (int(case["block_table"][b, pos // 16]), head, pos % 16)
    level = {0.0: 0, 2.0: 4, 1.0: 2, 12.0: 7, 24.0: 7}[score]
    channel = dim - 1 if channel is None else channel
    byte = case["cache"]["k_codes"][at + (channel // 2,)]
    keep = byte & (0x0f if channel % 2 else 0xf0)
    case["cache"]["k_codes"][at + (channel // 2,)] = keep | (level << 4 if channel % 2 else level)
    case["cache"]["k_scales"][at + (dim // 32 - 1,)] = {12.0: 128, 24.0: 129}.get(score, 127)


def _run(sv, case, **kw):
    g = Q.on_gpu(case)
    r = sv.kv_paged_attention_q4(*[g[n] for n in Q.NAMES], lse=True, scale=SCALE, **kw)
    torch.cuda.synchronize()
    return r["out"].cpu(), r["lse"].cpu()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256, 96])
@pytest.mark.parametrize("heads,kv,hint", [(2, 2, 0), (4, 2, 4), (8, 2, 12), (8, 2, 60)])
@pytest.mark.parametrize("split", [False, True])
def test_a_later_token_s_key(sv, heads, kv, hint, dim, dtype, split):
    """One key, seen by the last tokens alone, changes from an ordinary one to one that
    moves their references."""
    case = _case(heads, kv, dim, dtype, split, seed=dim)
    base = _run(sv, case, max_new=hint)
    lens, cu = case["seq_lens"].tolist(), case["cu_tokens"].tolist()
    for first in (1, 4, 6):             # the first token that sees it
        for score in (12.0, 24.0):
            for b, L in enumerate(lens):
                _set(case, b, L - NEW + first, dim, score)
            out, lse = _run(sv, case, max_new=hint)
            for b, L in enumerate(lens):
                _set(case, b, L - NEW + first, dim, 0.0)
                rows = slice(cu[b], cu[b] + first)
                assert torch.equal(lse[rows], base[1][rows]), (first, score, b)
                assert torch.equal(out[rows], base[0][rows]), (first, score, b)
                seen = slice(cu[b] + first, cu[b + 1])
                assert (lse[seen] > base[1][seen] + 0.5).all(), (first, score, b)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256, 96])
@pytest.mark.parametrize("split", [False, True])
def test_another_head_s_score(sv, split, dim, dtype):
    """A key that is large against one head's queries and does not change the others'
    scores (their queries are 0 in its channel)."""
    case = _case(8, 2, dim, dtype, split, seed=dim + 1)
    case["q"][:, 2, dim - 2] = 1.0
    base = _run(sv, case)
    for score in (12.0, 24.0):
        for b, L in enumerate(case["seq_lens"].tolist()):
            _set(case, b, L - NEW, dim, score, channel=dim - 2)
        out, lse = _run(sv, case)
        assert (lse[:, 2] > base[1][:, 2] + 0.5).all()
        others = [h for h in range(8) if h != 2]
        assert torch.equal(lse[:, others], base[1][:, others]), score
        assert torch.equal(out[:, others], base[0][:, others]), score


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256, 96])
@pytest.mark.parametrize("split", [False, True])
def test_a_neighbour_that_is_not_a_number(sv, split, dim, dtype):
    """The last token's references move in a later unit, or its queries are not a
    number."""
    case = _case(4, 2, dim, dtype, split, seed=dim + 2)
    for b, L in enumerate(case["seq_lens"].tolist()):
        _set(case, b, L - 1, dim, 24.0)
    base = _run(sv, case)
    for bad in (math.nan, math.inf):
        dirty = {**case, "q": case["q"].clone()}
        hit = torch.zeros(base[1].shape, dtype=torch.bool)
        for t in case["cu_tokens"].tolist()[:-1]:
            dirty["q"][t + NEW - 1, :, 3] = bad
            hit[t + NEW - 1] = True
        out, lse = _run(sv, dirty)
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
        assert torch.equal(lse[~hit], base[1][~hit]) and torch.equal(out[~hit], base[0][~hit]), bad
