"""What kv_paged_attention_q4 gives where products or values leave float32."""

import math

import pytest
import torch

from tests import kvcases as C
from tests import kvq4cases as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


def _run(sv, case, **kw):
    g = Q.on_gpu(case)
    r = sv.kv_paged_attention_q4(*[g[n] for n in Q.NAMES], lse=True, **kw)
    torch.cuda.synchronize()
    return r["out"].cpu(), r["lse"].cpu()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256, 96])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_value_leaves_the_lse(sv, dim, dtype, bad):
    case = Q.attend_case([40, 6000], [9, 2], 4, 2, dim, 16, dtype, seed=50)
    out, lse = _run(sv, case)
    for b, pos in ((0, 3), (0, 44), (1, 2000)):
        case["cache"]["v_scales"][int(case["block_table"][b, pos // 16]), 1, pos % 16] = bad
    got, got_lse = _run(sv, case)
    assert torch.equal(got_lse, lse)
    assert torch.isnan(got[:, 2:]).all() and torch.equal(got[:, :2], out[:, :2])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256, 96])
@pytest.mark.parametrize("every", [1, 3])
@pytest.mark.parametrize("ctx", [50, 700, 9000])
def test_products_beyond_float32(sv, ctx, every, dim, dtype):
    """Keys of 6 * 2^127 in 32 channels at every first or third position, 0 elsewhere, all
    values 1: against -4 they have no weight, against 4 the row is not a number,
    against 0 they score 0."""
    L, new = ctx + 2, 2
    n = -(-L // 16)
    cache = dict(k_codes=torch.zeros((n, 1, 16, dim // 2), dtype=torch.uint8),
                 k_scales=torch.full((n, 1, 16, -(-dim // 128) * 4), 127, dtype=torch.uint8),
                 v_codes=torch.full((n, 1, 16, dim // 2), 0x22, dtype=torch.uint8),
                 v_scales=torch.ones((n, 1, 16)))
    t = torch.arange(0, n * 16, every)
    cache["k_codes"][t // 16, 0, t % 16, :16] = 0x77
    cache["k_scales"][t // 16, 0, t % 16, 0] = 254
    q = torch.zeros((new, 3, dim), dtype=C.DT[dtype])
    q[:, 0, :32], q[:, 1, :32] = -4.0, 4.0
    case = dict(q=q, cache=cache, block_table=torch.arange(n, dtype=torch.int32)[None],
                seq_lens=torch.tensor([L], dtype=torch.int32),
                cu_tokens=torch.tensor([0, new], dtype=torch.int32))
    out, lse = _run(sv, case)
    for j in range(new):
        sees = ctx + j + 1
        left = sees - -(-sees // every)
        assert torch.isnan(out[j, 1]).all() and torch.isnan(lse[j, 1])
        assert (out[j, 2] == 1.0).all() and abs(lse[j, 2].item() - math.log(sees)) < 1e-5
        if left:
            assert (out[j, 0] == 1.0).all() and abs(lse[j, 0].item() - math.log(left)) < 1e-5
        else:
            assert (out[j, 0] == 0.0).all() and lse[j, 0].item() == -math.inf
