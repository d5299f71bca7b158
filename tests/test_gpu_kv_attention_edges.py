"""GPU parity of kv_paged_attention at calls that its other tests leave out, within
bounds by arithmetic (tests/kvcases.py)."""

import pytest
import torch

from tests import kvcases as C

pytestmark = pytest.mark.gpu

NAMES = ("q", "k_cache", "v_cache", "block_table", "seq_lens", "cu_tokens")


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


@pytest.mark.parametrize("ctx,new,heads,dim,dtype,hint", [
    (60, 140, 256, 64, "bf16", 1),       # 5 tiles of 32 rows for 4 places a head
    (10, 200, 128, 128, "f16", 1),       # 7 for 6
    (70, 160, 64, 64, "f32", 0),         # 40 tiles of 4 rows for 16
    (1, 40, 128, 248, "f32", 0),         # 20 of 2 for 8
    (9, 150, 256, 256, "bf16", 0)])      # 3 tiles of 64 rows for 2
def test_one_sequence_of_more_tiles_than_places(sv, ctx, new, heads, dim, dtype, hint):
    """A single sequence whose tiles alone fill the chip, on a table so wide that its
    keys could be split."""
    case = C.attend_case([ctx], [new], heads, heads, dim, 16, dtype, seed=31)
    wide = torch.full((1, 600), -1, dtype=torch.int32)
    wide[:, :case["block_table"].shape[1]] = case["block_table"]
    g = C.on_gpu({**case, "block_table": wide})
    r = sv.kv_paged_attention(*[g[n] for n in NAMES], lse=True, max_new=hint)
    torch.cuda.synchronize()
    assert r["workspace"] is not None
    C.check(C.to64(r["out"]), C.to64(r["lse"]), C.reference(case), dtype, dim)
